// sv_head_host.h -- host-side argument checks, piece sizes and workspace layouts
// of the vocabulary-head operators, in plain C++ with no HIP (a CPU build with
// sanitizers drives it over valid and invalid shapes).
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_head.h"

namespace sv_head_host {

constexpr int TOP = 32;                  // stored entries per row (sv_head_kd)
constexpr int STEP = 128;                // bytes of k per step of the tiled product
constexpr int CUS = 256;                 // compute units of the GPU
constexpr int64_t PIECE = (int64_t)512 << 20;   // bytes of a piece's dz and weight
// least steps of a workgroup of the hidden gradient (24 rows of 1024 x 20000 56 us with 8,
// 54 with 4, whose sums ride with dW; 5 of 72 x 53559 49.0 and 50.4)
constexpr int RUN = 4;
// A launch holds fewer than 2^32 work items in a dimension: rows (of at most 256 work
// items) a launch, and the largest number of workgroups of `threads`.
constexpr int64_t MAX_ROWS = (int64_t)1 << 23;
constexpr int64_t max_groups(int threads) { return 0xffffffffLL / threads; }
constexpr int64_t MAX_LD = (int64_t)1 << 22;   // bytes between rows of a tiled operand: a tile's offsets fit 31 bits

inline int64_t cdiv(int64_t x, int64_t m);
inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
// bytes between rows of n bytes: an odd number of 128-byte lines, so that rows
// spread over the L2's channels
inline int64_t spread(int64_t n) { return (cdiv(n, 128) | 1) * 128; }
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
inline int esize(int dtype) { return dtype == SV_F32 ? 4 : dtype == SV_BF16 ? 2 : 1; }
// Tiles of 256 x 256 instead of 128 x 128: they read each operand half as often (190 rows
// of 4096 x 151936: 8-bit logits 214 to 199 us, cross entropy 1740 to 1510), but where
// those of 128, two a CU, are one round, they would leave CUs without one (250 rows of
// 1024 x 32000, 125 tiles: 24 to 21 and 164 to 140; 250 of 4096 x 8000: 48 to 30 and 247
// to 165), and 128 rows or fewer are one row of the smaller tiles.
inline bool large_tiles(int64_t N, int64_t V) { return N > 128 && cdiv(N, 128) * cdiv(V, 128) > 2 * CUS; }
inline bool real_dtype(int dt) { return dt == SV_F32 || dt == SV_BF16; }

// ------------------------------------------------------------------- 8-bit rows
inline int check_act8(int N, int H, int dtype, const void *x, int64_t x_stride, const void *codes,
                      int64_t codes_stride, const void *scale) {
  if (!real_dtype(dtype)) return SV_ERR_DTYPE;
  if (N < 0 || H < 1 || H > SV_HEAD_MAX_H) return SV_ERR_SHAPE;
  if ((x_stride && x_stride < H) || (codes_stride && codes_stride < H)) return SV_ERR_SHAPE;
  if (N && (!x || !codes || !scale)) return SV_ERR_NULL;
  return SV_OK;
}

// ---------------------------------------------------------------- 8-bit logits
// Copied operands (rows that are not made of whole aligned steps) have rows of Kp bytes.
struct LogitsLayout {
  int64_t Kp;
  int64_t piece;                         // vocabulary entries per product where the weight is copied
  size_t codes, scale, weight, total;
};

inline bool logits_shape_ok(const sv_logits_shape_t *s) {
  if (s->N < 0 || s->H < 1 || s->H > SV_HEAD_MAX_H || s->V < 1 || s->V > SV_HEAD_MAX_V) return false;
  if (s->hidden_dtype != SV_I8 && !real_dtype(s->hidden_dtype)) return false;
  if (!real_dtype(s->out_dtype)) return false;
  if ((s->hidden_stride && s->hidden_stride < s->H) || (s->weight_stride && s->weight_stride < s->H) ||
      (s->out_stride && s->out_stride < s->V))
    return false;
  // one launch of whichever tiles (more would be logits of 500 GB)
  return cdiv(s->N, 128) * cdiv(s->V, 128) <= max_groups(256) && cdiv(s->N, 256) * cdiv(s->V, 256) <= max_groups(512);
}

// Whether weight code rows can be read in 16-byte pieces where they lie.
inline bool logits_direct(int64_t stride, uintptr_t base) { return stride % 16 == 0 && stride <= MAX_LD && base % 16 == 0; }

inline LogitsLayout logits_layout(const sv_logits_shape_t *s) {
  LogitsLayout L;
  L.Kp = up(s->H, STEP);
  // a copied piece of about 128 MB: it stays in the 256 MB Infinity Cache between its copy and its product
  L.piece = up(((int64_t)128 << 20) / L.Kp, 256);
  if (L.piece > up(s->V, 256)) L.piece = up(s->V, 256);
  size_t o = 0;
  L.codes = o;  o = up(o + (size_t)s->N * L.Kp, 256);
  L.scale = o;  o = up(o + (size_t)s->N * 4, 256);
  L.weight = o; o = up(o + (size_t)L.piece * L.Kp, 256);
  L.total = o;
  return L;
}

inline int check_logits(const sv_logits_shape_t *s, const void *hidden, const void *hidden_scale, const void *codes,
                        const void *wscale, const void *logits, const void *ws, size_t wsb, bool *nothing) {
  *nothing = false;
  if (!s) return SV_ERR_NULL;
  if ((s->hidden_dtype != SV_I8 && !real_dtype(s->hidden_dtype)) || !real_dtype(s->out_dtype)) return SV_ERR_DTYPE;
  if (!logits_shape_ok(s)) return SV_ERR_SHAPE;
  if (s->N == 0) { *nothing = true; return SV_OK; }
  if (!hidden || !codes || !wscale || !logits || (s->hidden_dtype == SV_I8 && !hidden_scale)) return SV_ERR_NULL;
  if (!ws || wsb < logits_layout(s).total || ((uintptr_t)ws & 255)) return SV_ERR_WORKSPACE;
  return SV_OK;
}

// ------------------------------------------------------------------------ losses
struct Plan {
  int e;                                 // bytes of an element
  int64_t Kp;                            // hidden width in whole steps, elements
  int64_t Np;                            // rows in whole steps, elements
  int64_t piece, pieces;                 // vocabulary entries per piece, pieces
  int64_t x_ld, dz_ld;                   // bytes between copied rows (of hidden and weight), rows of dz
  int64_t xw_ld, dzw_ld;                 // the same for dW's operands, rows of 16-byte blocks
  int bm, bn;                            // tile of the products
  bool keep;                             // the forward product's logits stay in dz (fp32, one piece)
  int terms;                             // bf16 terms of dz in rows of their own (beyond bm = 32, whose tiles hold two)
  bool narrow;                           // tiles of 64 columns against the weight's rows
  // the hidden gradient: chunks of a piece, steps of one; workgroups, tiles each may touch
  int chunks, full, groups, slots;
  // workspace sections
  size_t counts, perm, alpha, ga, lse2, w, flags, zt, pt, term, part, xs, xw, dz, dzw, wt, acc, total;
};

inline bool head_shape_ok(const sv_head_shape_t *s, bool kd) {
  if (s->N < 0 || s->N > SV_HEAD_MAX_N || s->H < 1 || s->H > SV_HEAD_MAX_H || s->V < 1 || s->V > SV_HEAD_MAX_V)
    return false;
  if (!real_dtype(s->dtype) || (s->hidden_dtype != s->dtype && s->hidden_dtype != SV_I8)) return false;
  if (s->grads & ~(SV_GRAD_HIDDEN | SV_GRAD_WEIGHT | SV_GRAD_TWO_TERMS) || s->grads == SV_GRAD_TWO_TERMS) return false;
  if ((s->hidden_stride && s->hidden_stride < s->H) || (s->weight_stride && s->weight_stride < s->H)) return false;
  if (kd) {
    if (s->temperature != 1.f) return false;
    if (s->N > 0 && (s->S < 1 || s->group < 1 || s->S % s->group != 0)) return false;
    if (!(s->w_max > 0.f)) return false;
  }
  return true;
}

// Whether the weight's rows are whole aligned steps where they lie.
inline bool weight_direct(const sv_head_shape_t *s, uintptr_t base) {
  const int64_t e = esize(s->dtype), ld = (s->weight_stride ? s->weight_stride : s->H) * e;
  return (s->H * e) % STEP == 0 && ld % 16 == 0 && ld <= MAX_LD && base % 16 == 0;
}

// direct: the weight is read where it lies, else copied a piece at a time.
inline Plan plan_for(const sv_head_shape_t *s, bool kd, bool direct) {
  Plan p;
  const int e = p.e = esize(s->dtype), q = STEP / e;
  const int64_t N = s->N, H = s->H, T = kd ? TOP : 1;
  p.Kp = up(H, q);
  p.Np = up(N, q);
  p.bm = N <= 32 ? 32 : s->dtype == SV_F32 ? 64 : large_tiles(N, s->V) ? 256 : 128;
  p.bn = p.bm == 32 ? 128 : p.bm;
  p.narrow = p.bm == 32 && s->V < 2 * CUS * 128;
  // A piece: its dz, for dx and for dW, and a copied weight take PIECE bytes together;
  // a whole number of 256 entries, all pieces alike.  More pays a little (4096 rows,
  // 4096 x 151936 in bf16, with the weight counted too: 13.2 ms with 256 MB, 12.8 with
  // 640, 12.6 with 1280, for fewer passes over the sums of dx and fewer last rounds of
  // tiles), but the logits in fp32 would be 2.5 GB.
  p.terms = (s->grads & SV_GRAD_TWO_TERMS) && s->dtype == SV_BF16 && p.bm > 32 ? 2 : 1;
  int64_t per = (s->grads ? 2 * p.terms * p.Np * e : 0) + (direct ? 0 : p.Kp * e);
  if (per < 16) per = 16;
  int64_t most = PIECE / per / 256 * 256;
  if (most < 256) most = 256;
  const int64_t by_ld = MAX_LD / 16 - 8;           // rows of blocks (and a line more)
  if (most > by_ld) most = by_ld;
  p.pieces = cdiv(s->V, most);
  p.piece = up(cdiv(s->V, p.pieces), 256);
  p.pieces = cdiv(s->V, p.piece);
  p.keep = s->grads && s->dtype == SV_F32 && p.pieces == 1;
  // the hidden gradient.  Workgroups: as many as run at once (LDS: one tile of 256, two
  // of 128 or 32, four of 64 rows a CU), fewer where a run would be short.  Chunks: no
  // more than workgroups share a tile (4096 rows of 4096 x 151936 in eight: 3220 to 3820
  // us, for the sums)
  const int64_t tiles = cdiv(N < 1 ? 1 : N, p.bm) * cdiv(H, p.bn), steps = p.piece * e / STEP;
  const int64_t most_groups = CUS * (p.bm == 256 ? 1 : p.bm == 64 ? 4 : 2), g = cdiv(tiles * steps, RUN);
  p.groups = (int)(g < most_groups ? g < 1 ? 1 : g : most_groups);
  p.chunks = 1;
  while (p.chunks < 8 && 2 * p.chunks * tiles <= p.groups) p.chunks *= 2;
  p.groups -= p.groups % p.chunks;
  p.full = (int)cdiv(steps, p.chunks);
  const int64_t run = cdiv(tiles * p.full, p.groups / p.chunks);
  p.slots = (int)(cdiv(run > RUN ? run : RUN, p.full) + 1);
  const bool gh = s->grads & SV_GRAD_HIDDEN, gw = s->grads & SV_GRAD_WEIGHT;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = (o + bytes + 255) & ~(size_t)255; return at; };
  p.counts = take(256);
  p.perm = take(N * 4);
  p.alpha = take(N * 4);
  p.ga = take(N * 4);
  p.lse2 = take(N * 4);
  p.w = take(N * 4);
  p.flags = take(N * 4);
  p.zt = take(N * T * 4);
  p.pt = take(kd ? N * T * 4 : 0);
  p.term = take(N * 8);
  p.part = take((size_t)cdiv(s->V, p.narrow || p.bm == 64 ? 64 : 128) * N * 8);
  p.x_ld = spread(p.Kp * e);
  p.dz_ld = spread(p.piece * e);
  p.xs = take((size_t)p.Np * p.x_ld);
  p.xw_ld = spread(p.Kp * 16);
  p.dzw_ld = spread(p.piece * 16);
  p.xw = take(gw ? (size_t)(p.terms * p.Np * e / 16) * p.xw_ld : 0);
  p.dz = take(gh || p.keep ? (size_t)(p.terms * p.Np) * p.dz_ld : 0);
  p.dzw = take(gw ? (size_t)(p.terms * p.Np * e / 16) * p.dzw_ld : 0);
  p.wt = take(direct ? 0 : (size_t)p.piece * p.x_ld);
  p.acc = take(gh ? (size_t)p.groups * p.slots * p.bm * p.bn * 4 : 0);
  p.total = o;
  return p;
}

// Vocabulary entries of one launch of the forward product, whose tiles are mt x (a
// column of `bn` entries), `threads` each: whole tiles of 256.  (450,000 rows of fp32 x
// 151936 are 2^32 work items.)
inline int64_t launch_columns(int64_t mt, int bn, int threads) { return max_groups(threads) / mt * bn / 256 * 256; }

// What a call may need: the copying plan where the weight's address decides.
inline size_t head_bytes(const sv_head_shape_t *s, bool kd) {
  const size_t copied = plan_for(s, kd, false).total;
  if (!weight_direct(s, 0)) return copied;
  const size_t direct = plan_for(s, kd, true).total;
  return direct > copied ? direct : copied;
}

inline int check_head(const sv_head_shape_t *s, bool kd, const void *hidden, const void *hidden_scale,
                      const void *weight, const void *a, const void *b, const void *c, const void *d, const void *rows,
                      const void *loss, const void *gh, const void *gw, const void *ws, size_t wsb, bool *nothing) {
  *nothing = false;
  if (!s) return SV_ERR_NULL;
  if (!real_dtype(s->dtype) || (s->hidden_dtype != s->dtype && s->hidden_dtype != SV_I8)) return SV_ERR_DTYPE;
  if (!(s->temperature > 0.f) || s->temperature == INFINITY) return SV_ERR_TEMPERATURE;
  if (!head_shape_ok(s, kd)) return SV_ERR_SHAPE;
  if (s->N == 0) { *nothing = true; return SV_OK; }
  if (!hidden || !weight || !a || !rows || !loss || (s->hidden_dtype == SV_I8 && !hidden_scale)) return SV_ERR_NULL;
  if (kd && (!b || !c || !d)) return SV_ERR_NULL;
  if (((s->grads & SV_GRAD_HIDDEN) && !gh) || ((s->grads & SV_GRAD_WEIGHT) && !gw)) return SV_ERR_NULL;
  if (!ws || wsb < head_bytes(s, kd) || ((uintptr_t)ws & 255)) return SV_ERR_WORKSPACE;
  return SV_OK;
}

}  // namespace sv_head_host
