// sv_logprobs_host.h -- host-side argument checks and plans of the log-probability
// operators, in plain C++ with no HIP (a CPU build with sanitizers drives it over valid
// and invalid shapes).
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"
#include "sv_head_host.h"
#include "sv_logprobs.h"

namespace sv_logprobs_host {

using sv_head_host::cdiv;
using sv_head_host::esize;
using sv_head_host::real_dtype;

constexpr int VECS = 4;                  // 16-byte vectors of a thread at a time
constexpr int LIST = 32;                 // alternatives that a list holds
// a launch holds every shape's workgroups: one a row, or at most 64 each of fewer than 128 rows
static_assert(SV_HEAD_MAX_N <= sv_head_host::max_groups(1024) && 128 * 64 <= sv_head_host::max_groups(1024), "one launch");

// A row's share of the launch: waves of a workgroup, workgroups of a row.
struct Plan {
  int waves, parts;
  int64_t batch, batches;                // entries of a workgroup's step, steps of a row
  size_t stats, keys, total;             // workspace sections (parts > 1)
};

inline Plan plan_for(const sv_logprobs_shape_t *s) {
  Plan p;
  const int64_t w = 16 / esize(s->dtype);
  // Few rows are cut into parts, joined in a launch of their own, where a row is more than
  // three steps of 16 waves (that launch costs the host 3 us too): into many small ones without
  // alternatives, into fewer with them, whose lists take longer to join.  Rows of 151936 bf16, cut
  // and uncut: one 7.1 and 16 us, 64 11.4 and 18.7, 127 17.1 and 19.2, 192 21.7 and 20.7, 256
  // 24.3 and 21.4; with twenty alternatives one 16.3 and 20.6, 64 18.7 and 24.3, 127 23.5 and
  // 25.2, 192 26.7 and 26.3.  The border at 128 rows is lower than these put it (128 to 160 rows
  // would gain a tenth to a twentieth), and rows that begin a second round on 256 CUs would gain
  // from a cut as well (300 27.6 and 35.5).  From 1024 rows on four waves a row fill the chip.
  const int64_t N = s->N < 1 ? 1 : s->N, step = 16 * 64 * VECS * w;
  const bool cut = N < 128 && s->V > 3 * step;
  p.waves = (cut && !s->top) || N >= 1024 ? 4 : 16;
  p.batch = (int64_t)p.waves * 64 * VECS * w;
  p.batches = cdiv(s->V, p.batch);
  p.parts = 1;
  if (cut && p.batches > 2) {
    const int64_t most = p.waves == 4 ? cdiv(1024, N) : 256 / N, by = cdiv(p.batches, 2);
    p.parts = (int)(most < by ? most : by);
    if (p.parts > 64) p.parts = 64;
  }
  const size_t n = p.parts > 1 ? (size_t)s->N * p.parts : 0;
  p.stats = 0;
  p.keys = (n * 24 + 255) & ~(size_t)255;
  p.total = p.keys + (s->top ? n * LIST * 8 : 0);
  return p;
}

inline bool temperature_ok(float t) { return t > 0.f && t < INFINITY && 1.44269504f / t < INFINITY; }

inline bool shape_ok(const sv_logprobs_shape_t *s) {
  return s->N >= 0 && s->N <= SV_HEAD_MAX_N && s->V >= 1 && s->V <= SV_HEAD_MAX_V && real_dtype(s->dtype) &&
         s->top >= 0 && s->top <= SV_LOGPROBS_MAX_TOP && (!s->row_stride || s->row_stride >= s->V);
}

inline int check(const sv_logprobs_shape_t *s, const void *logits, const void *tokens, const void *logp,
                 const void *top_logp, const void *top_idx, const void *ws, size_t wsb, bool *nothing) {
  *nothing = false;
  if (!s) return SV_ERR_NULL;
  if (!real_dtype(s->dtype)) return SV_ERR_DTYPE;
  if (!temperature_ok(s->temperature)) return SV_ERR_TEMPERATURE;
  if (!shape_ok(s)) return SV_ERR_SHAPE;
  if (s->N == 0) { *nothing = true; return SV_OK; }
  if (!logits || !tokens || !logp || (s->top && (!top_logp || !top_idx))) return SV_ERR_NULL;
  const size_t need = plan_for(s).total;
  if (need && (!ws || wsb < need || ((uintptr_t)ws & 255))) return SV_ERR_WORKSPACE;
  return SV_OK;
}

inline int check_grad(const sv_logprobs_grad_shape_t *s, const void *logits, const void *tokens, const void *norm,
                      const void *entropy, const void *grad_logp, const void *grad_entropy, const void *grad,
                      bool *nothing) {
  *nothing = false;
  if (!s) return SV_ERR_NULL;
  if (!real_dtype(s->dtype) || !real_dtype(s->grad_dtype)) return SV_ERR_DTYPE;
  if (!temperature_ok(s->temperature)) return SV_ERR_TEMPERATURE;
  if (s->N < 0 || s->N > SV_HEAD_MAX_N || s->V < 1 || s->V > SV_HEAD_MAX_V || (s->row_stride && s->row_stride < s->V) ||
      (s->grad_stride && s->grad_stride < s->V))
    return SV_ERR_SHAPE;
  if (s->N == 0) { *nothing = true; return SV_OK; }
  if (!logits || !tokens || !norm || !grad_logp || !grad || (grad_entropy && !entropy)) return SV_ERR_NULL;
  const int64_t rs = s->row_stride ? s->row_stride : s->V, gs = s->grad_stride ? s->grad_stride : s->V;
  if (logits == grad && (rs != gs || s->dtype != s->grad_dtype)) return SV_ERR_SHAPE;
  return SV_OK;
}

}  // namespace sv_logprobs_host
