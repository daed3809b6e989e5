// sv_mx4_host.h -- host-side argument checks, plans and workspace layouts of the 4-bit rows
// and head logits, in plain C++ with no HIP (a CPU build with sanitizers drives it over
// valid and invalid shapes).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_head_host.h"
#include "sv_mx4.h"

namespace sv_mx4_host {

using sv_head_host::cdiv;
using sv_head_host::CUS;
using sv_head_host::esize;
using sv_head_host::MAX_LD;
using sv_head_host::real_dtype;
using sv_head_host::up;

constexpr int BLOCK = SV_MX4_BLOCK;
constexpr int SPAN = 256;                // bytes of k of the tiled product's unrolled pair of steps
constexpr int64_t LDS_ROWS = 160 << 10;  // bytes of hidden rows that a workgroup may hold

inline int64_t code_bytes(int64_t H) { return cdiv(H, 2); }
inline int64_t blocks(int64_t H) { return cdiv(H, BLOCK); }

inline int check_rows(int N, int H, int dtype, const void *x, int64_t x_stride, const void *codes, int64_t codes_stride,
                      const void *scale, int64_t scale_stride) {
  if (!real_dtype(dtype)) return SV_ERR_DTYPE;
  if (N < 0 || H < 1 || H > SV_HEAD_MAX_H) return SV_ERR_SHAPE;
  if ((x_stride && x_stride < H) || (codes_stride && codes_stride < code_bytes(H)) ||
      (scale_stride && scale_stride < blocks(H)))
    return SV_ERR_SHAPE;
  if (N && (!x || !codes || !scale)) return SV_ERR_NULL;
  return SV_OK;
}

// How a call goes: the hidden rows held by every workgroup in LDS, each of its waves
// streaming the weight's rows from memory to registers; or tiles of both operands.
struct Plan {
  bool held;
  int frags;                             // held: fragments of 16 hidden rows
  bool fused;                            // held: every workgroup forms the hidden rows' codes itself
  int64_t nks;                           // held: 128-element steps of k
  int64_t image, x_scales;               // bytes of the hidden rows' codes and scales, as staged
  int64_t Kp, x_ld;                      // tiles: bytes of a staged code row, and between two
  int64_t groups;                        // tiles: 16-block groups of scales
  int64_t rows;                          // tiles: hidden rows that a launch stages, whole groups of scales
  bool large;                            // tiles of 256 x 256
  // tiles: vocabulary entries per product where the weight is copied, and where only its
  // scales are staged
  int64_t piece, scaled;
  size_t codes, scales, weight, wscale, total;
};

// The hidden rows' parts in LDS: their codes, then their scales.
inline int64_t held_bytes(int64_t N, int64_t H) {
  const int64_t nks = cdiv(H, 128);
  return N * (nks * 64 + cdiv(nks, 4) * 16);
}

inline bool shape_ok(const sv_logits4_shape_t *s) {
  if (s->N < 0 || s->H < 1 || s->H > SV_HEAD_MAX_H || s->V < 1 || s->V > SV_HEAD_MAX_V) return false;
  if (s->hidden_dtype != SV_MX4 && !real_dtype(s->hidden_dtype)) return false;
  if (!real_dtype(s->out_dtype)) return false;
  const int64_t row = s->hidden_dtype == SV_MX4 ? code_bytes(s->H) : s->H;
  if ((s->hidden_stride && s->hidden_stride < row) || (s->hidden_scale_stride && s->hidden_scale_stride < blocks(s->H)) ||
      (s->weight_stride && s->weight_stride < code_bytes(s->H)) ||
      (s->weight_scale_stride && s->weight_scale_stride < blocks(s->H)) || (s->out_stride && s->out_stride < s->V))
    return false;
  // one launch of whichever tiles (more would be logits of 500 GB)
  return cdiv(s->N, 128) * cdiv(s->V, 128) <= sv_head_host::max_groups(256);
}

// Where the tiled product's lanes take their scales.  Those of a row's 16 blocks are four words,
// blocks 4 k + q, k = 0 .. 3, in lane 16 q + row % 16's; a lane's words of four times 16 rows lie
// together.  So 64 rows are a group, and memory that begins with the first of one goes on as the
// whole's does.
constexpr int SCALE_ROWS = 64;
constexpr int64_t tiled_scale(int64_t row, int64_t group, int64_t lane, int64_t groups) {
  return ((row / SCALE_ROWS * groups + group) * 64 + lane) * 4 + row / 16 % 4;
}

// Whether weight code rows can be read in 16-byte pieces where they lie (what lies behind
// a row's end meets zeros of the hidden rows).
inline bool codes_direct(int64_t stride, uintptr_t base) { return stride % 16 == 0 && stride <= MAX_LD && base % 16 == 0; }

inline Plan plan_for(const sv_logits4_shape_t *s) {
  Plan p = {};
  const int64_t N = s->N, H = s->H;
  p.nks = cdiv(H, 128);
  // Held: up to 128 rows that LDS holds, but for those beyond 64 of a large vocabulary whose
  // results, which it stores 32 bytes at a time, count for much beside the weight, where tiles
  // can read that in place (128 rows of 512 x 151936 32.8 us and 23.9 in tiles, of 2048 47.7
  // and 42.7; 80 rows of 2048 x 151936 41.0 and 40.9, 128 of 1024 x 32000 13.2 and 13.7; 64 of
  // 1024 x 151936 25.4 and 27.5, 8 rows 17.0 and 23.8).  Measured at 32000 and 151936 entries;
  // where between them the border lies was not.
  const int64_t ld = s->weight_stride ? s->weight_stride : code_bytes(H);
  const bool tiles = N > 64 && s->V > 65536 && 24 * N > H && ld % 16 == 0;
  p.held = N <= 128 && held_bytes(N, H) <= LDS_ROWS && !tiles;
  p.frags = (int)cdiv(N, 16);
  if (p.frags == 0) p.frags = 1;
  if (p.frags == 7) p.frags = 8;
  p.fused = p.held && s->hidden_dtype != SV_MX4 && N <= 16 && N * H <= 16384;
  p.Kp = up(code_bytes(H), SPAN);
  p.groups = p.Kp / SPAN;
  p.rows = sv_head_host::max_groups(256) * 1024 / (p.Kp / 4) / SCALE_ROWS * SCALE_ROWS;
  p.large = sv_head_host::large_tiles(N, s->V);
  size_t o = 0;
  auto take = [&](int64_t bytes) { const size_t at = o; o = (o + bytes + 255) & ~(size_t)255; return at; };
  if (p.held) {
    p.image = N * p.nks * 64;
    p.x_scales = N * cdiv(p.nks, 4) * 16;
    p.codes = take(p.fused ? 0 : p.image);
    p.scales = take(p.fused ? 0 : p.x_scales);
    p.total = o;
    return p;
  }
  p.x_ld = sv_head_host::spread(p.Kp);
  p.image = N * p.x_ld;
  p.x_scales = up(N, 256) * p.groups * 16;
  // a copied piece of about 128 MB: it stays in the 256 MB Infinity Cache between its copy and its product
  p.piece = up(((int64_t)128 << 20) / p.x_ld, 256);
  if (p.piece > up(s->V, 256)) p.piece = up(s->V, 256);
  // staged scales of a piece: 256 MB at most, and a launch's worth
  p.scaled = ((int64_t)256 << 20) / (p.groups * 16) / 256 * 256;
  if (p.scaled > up(s->V, 256)) p.scaled = up(s->V, 256);
  p.codes = take(p.image);
  p.scales = take(p.x_scales);
  // (Copied rows have their place also where the stride is aligned: the address, which a size
  // must do for whatever it is, may not be, and such a weight is copied as well.)
  p.weight = take(p.piece * p.x_ld);
  p.wscale = take((p.scaled > p.piece ? p.scaled : p.piece) * p.groups * 16);
  p.total = o;
  return p;
}

inline int check_logits(const sv_logits4_shape_t *s, const void *hidden, const void *hidden_scale, const void *codes,
                        const void *wscale, const void *logits, const void *ws, size_t wsb, bool *nothing) {
  *nothing = false;
  if (!s) return SV_ERR_NULL;
  if ((s->hidden_dtype != SV_MX4 && !real_dtype(s->hidden_dtype)) || !real_dtype(s->out_dtype)) return SV_ERR_DTYPE;
  if (!shape_ok(s)) return SV_ERR_SHAPE;
  if (s->N == 0) { *nothing = true; return SV_OK; }
  if (!hidden || !codes || !wscale || !logits || (s->hidden_dtype == SV_MX4 && !hidden_scale)) return SV_ERR_NULL;
  const size_t need = plan_for(s).total;
  if (need && (!ws || wsb < need || ((uintptr_t)ws & 255))) return SV_ERR_WORKSPACE;
  return SV_OK;
}

}  // namespace sv_mx4_host
