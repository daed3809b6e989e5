// sv_logprobs.hip -- log-probabilities of given tokens with the rows' entropies and
// largest alternatives, and their gradient, for gfx950 (MI355X).
//
// One pass over the logits.  With the running maximum m of what a thread has read, c =
// log2(e) / T and y = (z - m) c, it keeps s = sum 2^y and a = sum 2^y y; a larger maximum M
// scales both by f = 2^((m - M) c), a -> f (a + s (m - M) c).  At the end ln s is the
// normaliser's part beyond the maximum, and ln s - ln 2 a / s the entropy.  Exponents are
// exact to their own rounding whatever the logits' magnitude (rows filled with the type's
// lowest value among them).
//
// Alternatives: a wave keeps the `top` best keys it has seen, a key holding value and
// index so that larger is better and no two are equal.  A vector of logits costs one
// comparison of its maximum, which the softmax needs anyway, with a border that at least
// `top` entries reach; what passes goes to a buffer in LDS, and a full buffer is sorted into
// the list, whose last key is the next border.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "sv_device.h"
#include "sv_logprobs.h"
#include "sv_logprobs_host.h"

namespace {

using namespace sv_dev;
using sv_logprobs_host::cdiv;
using sv_logprobs_host::LIST;
using sv_logprobs_host::VECS;

typedef uint64_t Key;                    // value's order, then the complement of the index; 0: none
typedef u32x4 u32x4_any __attribute__((aligned(2)));

constexpr float LOG2E = 1.44269504088896341f;
constexpr double LN2 = 0.69314718055994531;

struct LogprobsP {
  const char *z;
  int64_t z_ld;                          // bytes
  const int32_t *tokens;
  float *logp, *entropy, *lse, *norm;
  int32_t *status;
  float *top_logp;
  int32_t *top_idx;
  int32_t N, V, top, ignore, parts;
  int64_t batch, batches;
  float T;
  double *stats;                         // [N][parts][3]: maximum, s, a
  Key *keys;                             // [N][parts][LIST]
};

// s = sum 2^y and a = sum 2^y y of the entries seen, y = (z - m) c with their maximum m
struct Stat {
  float m;
  double s, a;
};

// x + y, relative to the larger maximum (NaN where either is)
__device__ __forceinline__ Stat join(const Stat &x, const Stat &y, float c) {
  Stat r;
  r.m = fmax_nan(x.m, y.m);
  auto part = [&](const Stat &t, double &s, double &a) {
    const float d = t.m - r.m, f = t.m == r.m ? 1.f : __builtin_amdgcn_exp2f(d * c);
    s = f > 0.f ? t.s * (double)f : 0.0;
    a = f > 0.f ? (t.m == r.m ? t.a : (t.a + t.s * (double)(d * c)) * (double)f) : 0.0;
  };
  double s, a;
  part(x, r.s, r.a);
  part(y, s, a);
  r.s += s;
  r.a += a;
  return r;
}

// Of all lanes: the common maximum first, then each lane's part scaled to it once, so that the
// sums are plain ones (the lanes' order is fixed).
__device__ __forceinline__ Stat wave_join(Stat v, float c) {
  Stat r;
  r.m = wave_max_f(v.m);
  const float d = v.m - r.m, f = v.m == r.m ? 1.f : __builtin_amdgcn_exp2f(d * c);
  const bool some = f > 0.f;             // (NaN and empty lanes: none)
  const double a = v.m == r.m ? v.a : v.a + v.s * (double)(d * c);
  r.s = wave_sum_d(some ? v.s * (double)f : 0.0);
  r.a = wave_sum_d(some ? a * (double)f : 0.0);
  return r;
}

// The order of floats as that of unsigned integers; -0 as +0.  Never 0 for a number.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ Key key_of(float v, uint32_t index) { return (Key)order_of(v) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// Keys of the 64 lanes in descending order (a bitonic sort: 21 exchanges).
__device__ __forceinline__ Key sort_wave(Key k) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));         // (what depends on it is formed here, not held throughout)
#pragma unroll
  for (int n = 2; n <= 64; n <<= 1)
#pragma unroll
    for (int j = n >> 1; j; j >>= 1) {
      const Key o = __shfl(k, lane ^ j);
      const bool larger = ((lane & j) == 0) == ((lane & n) == 0);
      k = (o > k) == larger ? o : k;
    }
  return k;
}
// The best LIST of two descending lists, in descending order: lanes 0 .. 31 hold the one,
// lanes 32 .. 63 the other.  Lanes 0 .. 31 are given the result.
__device__ __forceinline__ Key merge_lists(Key k) {
  const int lane = threadIdx.x & 63;
  const Key o = __shfl(k, 63 - lane);
  k = o > k ? o : k;
#pragma unroll
  for (int j = 16; j; j >>= 1) {
    const Key p = __shfl_xor(k, j);
    k = (p > k) == ((lane & j) == 0) ? p : k;
  }
  return k;
}

// The best keys that a wave has seen: lanes 0 .. 31 hold them in descending order, beside what
// has come since in a buffer.  Entries come in the order of their indices, so of equal ones
// those that came first stay.
struct Best {
  Key list;
  float border;                          // larger values are taken (at first those above -inf)
  int count;                             // keys in the buffer
  bool sorted;                           // whether any are in the list
  Key *buffer;                           // LIST keys in LDS, the wave's own

  __device__ __forceinline__ void start(Key *b) {
    list = 0;
    border = NEG_INF;
    count = 0;
    sorted = false;
    buffer = b;
  }
  __device__ __forceinline__ void flush(int top) {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    const Key k = lane < LIST ? list : lane - LIST < count ? buffer[lane - LIST] : 0;
    __builtin_amdgcn_wave_barrier();
    list = sort_wave(k);
    count = 0;
    sorted = true;
    const Key w = __shfl(list, top - 1); // the top-th best
    if (w) border = fmax_nan(border, value_of(w));
  }
  // one entry of each lane
  __device__ __forceinline__ void offer(float v, uint32_t index, int top) {
    uint64_t who = __ballot(v > border);
    while (who) {
      const int lane = threadIdx.x & 63, room = LIST - count;
      const int place = __popcll(who & (((Key)1 << lane) - 1)), n = __popcll(who);
      const bool mine = who >> lane & 1;
      if (mine && place < room) buffer[count + place] = key_of(v, index);
      count += n < room ? n : room;
      if (n <= room) break;
      flush(top);
      who = __ballot(mine && place >= room && v > border);
    }
  }
};

// A border from the lanes' maxima so far: of 64 groups of lanes (WAVES lanes each) the top-th
// largest maximum, cut to 16 bits, so that at least `top` entries reach it and few others do (of
// random rows 24 for 20, 44 for 32).  groups: 64 words in LDS, and one for the result.
template <int WAVES> __device__ __forceinline__ void raise_border(Best &b, float most, int top, uint32_t *groups) {
  static_assert(WAVES == 4 || WAVES == 16, "groups within a row of lanes");
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  uint32_t u = most > NEG_INF ? order_of(most) : 0;
  auto with = [&](uint32_t v) { u = v > u ? v : u; };
  with(dpp<0xb1, 0xf, 0xf>(u, u));       // lanes 1 and 2 apart
  with(dpp<0x4e, 0xf, 0xf>(u, u));
  if constexpr (WAVES == 16) {
    with(dpp<0x124, 0xf, 0xf>(u, u));    // turned by 4 and 8
    with(dpp<0x128, 0xf, 0xf>(u, u));
  }
  if (lane % WAVES == 0) groups[wid * (64 / WAVES) + lane / WAVES] = u;
  __syncthreads();
  if (wid == 0) {
    u = groups[lane];
    uint32_t at = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t t = at | 1u << bit;
      at = __popcll(__ballot(u >= t)) >= top ? t : at;
    }
    if (lane == 0) groups[64] = at;
  }
  __syncthreads();
  const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane((int)groups[64]);
  // the value below it (below 0 that is no zero)
  if (at > order_of(NEG_INF)) b.border = fmax_nan(b.border, value_of((Key)(at - (at == 0x80000000u ? 2 : 1)) << 32));
}

// A thread's vectors of one step: entries at `at` + s * 64 * waves * W; past `end` -inf.
template <int DT, int WAVES>
__device__ __forceinline__ void load_step(const char *row, int64_t at, int64_t end, u32x4 (&r)[VECS]) {
  constexpr int E = Fmt<DT>::E, W = Fmt<DT>::W;
  constexpr uint32_t NEG = DT == SV_BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
  for (int s = 0; s < VECS; ++s) {
    const int64_t e = at + (int64_t)s * (64 * WAVES * W);
    r[s] = u32x4{NEG, NEG, NEG, NEG};
    if (e + W <= end) r[s] = __builtin_nontemporal_load((const u32x4_any *)(row + e * E));
  }
#pragma unroll
  for (int s = 0; s < VECS; ++s) {
    const int64_t e = at + (int64_t)s * (64 * WAVES * W);
    if (e < end && e + W > end) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (DT == SV_BF16) {
          const int64_t x = e + 2 * q;
          if (x < end) r[s][q] = 0xff800000u | *(const uint16_t *)(row + x * 2);
          if (x + 1 < end) r[s][q] = (r[s][q] & 0xffffu) | (uint32_t)*(const uint16_t *)(row + x * 2 + 2) << 16;
        } else {
          if (e + q < end) r[s][q] = *(const uint32_t *)(row + (e + q) * 4);
        }
      }
    }
  }
}

// What a row's results are, from its statistics and best keys (lanes 0 .. 31 of the wave
// that calls).
__device__ __forceinline__ void finish(const LogprobsP &P, int64_t n, const Stat &t, Key best, float zt, bool bad) {
  const int lane = threadIdx.x & 63;
  int st = bad ? SV_HEAD_BAD_TARGET : 0;
  if (!(t.m == t.m)) st |= SV_HEAD_NAN;
  else if (t.m == -NEG_INF) st |= SV_HEAD_POSINF;
  else if (t.m == NEG_INF) st |= SV_HEAD_EMPTY;
  const double T = (double)P.T, ls = log(t.s);
  if (lane == 0) {
    const float none = __builtin_nanf("");
    const double logp = ((double)zt - (double)t.m) / T - ls, h = ls - t.a / t.s * LN2;
    P.logp[n] = st ? none : (float)(logp < 0.0 ? logp : 0.0);
    if (P.entropy) P.entropy[n] = st ? none : (float)(h > 0.0 ? h : 0.0);
    if (P.lse) P.lse[n] = st ? none : (float)((double)t.m / T + ls);
    if (P.norm) {
      P.norm[n] = st ? none : t.m;
      P.norm[P.N + n] = st ? none : (float)ls;
    }
    if (P.status) P.status[n] = st;
  }
  if (lane < P.top) {
    const double v = (((double)value_of(best) - (double)t.m) / T - ls);
    P.top_logp[n * P.top + lane] = st ? __builtin_nanf("") : best ? (float)(v < 0.0 ? v : 0.0) : NEG_INF;
    P.top_idx[n * P.top + lane] = st || !best ? -1 : (int32_t)~(uint32_t)best;
  }
}

__device__ __forceinline__ void left_out(const LogprobsP &P, int64_t n) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    P.logp[n] = 0.f;
    if (P.entropy) P.entropy[n] = 0.f;
    if (P.lse) P.lse[n] = 0.f;
    if (P.norm) P.norm[n] = P.norm[P.N + n] = 0.f;
    if (P.status) P.status[n] = 0;
  }
  if (tid < P.top) {
    P.top_logp[n * P.top + tid] = NEG_INF;
    P.top_idx[n * P.top + tid] = -1;
  }
}

// The lists of WAVES waves into one, in all waves' lanes: pairs, then pairs of pairs.
template <int WAVES> __device__ __forceinline__ Key join_lists(Key mine, Key (*lists)[LIST]) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  if (lane < LIST) lists[wid][lane] = mine;
#pragma unroll 1
  for (int n = 1; n < WAVES; n <<= 1) {
    __syncthreads();
    if (wid % (2 * n) == 0) {
      const Key k = merge_lists(lists[wid + (lane >= LIST ? n : 0)][lane % LIST]);
      if (lane < LIST) lists[wid][lane] = k;
    }
  }
  __syncthreads();
  return lists[0][lane % LIST];
}

// The waves' best keys into one list, in wave 0's lanes.  Few (the usual case): each goes to the
// place that the number of larger ones gives it.  Many: sorted lists are joined in pairs, then
// pairs of pairs.
template <int WAVES>
__device__ __forceinline__ Key join_best(Best &best, Key (*lists)[LIST], int32_t *counts, Key *all, int top) {
  constexpr int FEW = 256;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  if (best.sorted) {
    best.flush(top);
    if (lane < LIST) lists[wid][lane] = best.list;
    best.count = __popcll(__ballot(lane < top && best.list != 0));
  }
  if (lane == 0) counts[wid] = best.count;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int c = counts[w];
    before += w < wid ? c : 0;
    total += c;
  }
  if (total <= FEW) {
    if (lane < best.count) all[before + lane] = lists[wid][lane];
    if (tid < LIST) all[FEW + tid] = 0;
    if (tid < 8 && total + tid < FEW) all[total + tid] = 0;
    __syncthreads();
    if (tid < total) {
      const Key k = all[tid];
      int place = 0;
      for (int j = 0; j < total; j += 8) {   // (eight reads under way together; zeros behind the last)
#pragma unroll
        for (int i = 0; i < 8; ++i) place += all[j + i] > k;
      }
      if (place < LIST) all[FEW + place] = k;
    }
    __syncthreads();
    return all[FEW + lane % LIST];
  }
  if (!best.sorted) best.flush(top);
  return join_lists<WAVES>(best.list, lists);
}

template <int DT, int WAVES, bool TOP>
__global__ __launch_bounds__(64 * WAVES) void logprobs_kernel(LogprobsP P) {
  constexpr int W = Fmt<DT>::W;
  __shared__ Key lists[TOP ? WAVES : 1][LIST], all[TOP ? 256 + LIST : 1];
  __shared__ uint32_t groups[TOP ? 65 : 1];
  __shared__ int32_t counts[TOP ? WAVES : 1];
  __shared__ Stat stats[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int64_t n = blockIdx.x / P.parts;
  const int part = (int)(blockIdx.x - n * P.parts);
  const char *row = P.z + n * P.z_ld;
  const float c = LOG2E / P.T;
  // steps of the row in equal runs
  const int64_t b0 = part * P.batches / P.parts, b1 = (part + 1) * P.batches / P.parts;
  const int64_t end = b1 * P.batch < P.V ? b1 * P.batch : P.V;
  int64_t at = b0 * P.batch + (int64_t)tid * W;
  Stat t = {NEG_INF, 0.0, 0.0};
  // Whether the wave's entries ask for the careful way: masked ones (0 times -inf), or so large
  // that a product's rounding is no small part of an exponent.
  bool general = false;
  Best best;
  u32x4 r[VECS], next[VECS];
  load_step<DT, WAVES>(row, at, end, r);
  // the first loads go out before the token is known, also those of rows that are left out
  const int token = P.tokens[n];
  if (token == P.ignore) {
    if (part == 0) left_out(P, n);
    return;
  }
  const bool bad = token < 0 || token >= P.V;
  const float zt = wid == 0 && !bad ? load_elem<DT>(row, token) : 0.f;
  if constexpr (TOP) best.start(lists[wid]);
  for (int64_t b = b0; b < b1; ++b, at += P.batch) {
    if (b + 1 < b1) load_step<DT, WAVES>(row, at + P.batch, end, next);
    float top[VECS], most = NEG_INF;
#pragma unroll
    for (int s = 0; s < VECS; ++s) {
      top[s] = unpack<DT>(r[s], 0);
#pragma unroll
      for (int w = 1; w < W; ++w) top[s] = fmax_nan(top[s], unpack<DT>(r[s], w));
      most = fmax_nan(most, top[s]);
    }
    const float m = fmax_nan(t.m, most);
    if (m != t.m) {                      // (NaN too)
      t = join(t, Stat{m, 0.0, 0.0}, c);
    }
    const float ref = m == NEG_INF ? 0.f : m, rc = ref * c;
    // (each pass unpacks its entries again: held unpacked they would take 32 registers)
#pragma unroll
    for (int s = 0; s < VECS; ++s) asm volatile("" : "+v"(r[s]));
    float s1 = 0.f, a1 = 0.f;
    general |= (b + 1) * P.batch > end;  // (what fills the last step is -inf)
    if (!general) {
      // one fused step an exponent; rc's rounding, the same for all, is taken out of the sums
#pragma unroll
      for (int s = 0; s < VECS; ++s)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float y = fmaf(unpack<DT>(r[s], w), c, -rc), e = __builtin_amdgcn_exp2f(y);
          s1 += e;
          a1 = fmaf(e, y, a1);           // (NaN where an entry is -inf)
        }
      const float lo = fmaf(ref, c, -rc);
      if (__ballot(!(a1 == a1) || !(fabsf(rc) <= 65536.f))) {
        general = true;
      } else {
        const double k = (double)__builtin_amdgcn_exp2f(-lo);
        t.s += (double)s1 * k;
        t.a += (double)fmaf(-lo, s1, a1) * k;
      }
    }
    if (general) {
#pragma unroll
      for (int s = 0; s < VECS; ++s) asm volatile("" : "+v"(r[s]));
      s1 = a1 = 0.f;
#pragma unroll
      for (int s = 0; s < VECS; ++s)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float y = __builtin_fmaxf((unpack<DT>(r[s], w) - ref) * c, -1e4f), e = __builtin_amdgcn_exp2f(y);
          s1 += e;
          a1 = fmaf(e, y, a1);
        }
      t.s += (double)s1;
      t.a += (double)a1;
    }
    if constexpr (TOP) {
      // (again after 2, 4, 8 .. steps: 256 rows of 151936 fp32 with twenty alternatives 40.6 us to
      // 36.0, without any 27.9)
      if (((b - b0) & (b - b0 + 1)) == 0) raise_border<WAVES>(best, m, P.top, groups);
#pragma unroll
      for (int s = 0; s < VECS; ++s) {
        // few lanes' vectors have an entry to take: each of those is spread over the lanes
        uint64_t who = __ballot(top[s] > best.border);
        while (who) {
          const int l = __builtin_ctzll(who);
          who &= who - 1;
          const uint32_t u0 = readlane(r[s][0], l), u1 = readlane(r[s][1], l), u2 = readlane(r[s][2], l),
                         u3 = readlane(r[s][3], l);
          const int q = DT == SV_BF16 ? lane >> 1 : lane;
          uint32_t u = q & 2 ? (q & 1 ? u3 : u2) : (q & 1 ? u1 : u0);
          if constexpr (DT == SV_BF16) u = lane & 1 ? u & 0xffff0000u : u << 16;
          const int64_t i = at + (int64_t)s * (64 * WAVES * W) + (int64_t)(l - lane) * W;
          best.offer(lane < W ? __uint_as_float(u) : NEG_INF, (uint32_t)i + lane, P.top);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < VECS; ++s) r[s] = next[s];
  }
  t = wave_join(t, c);
  Key k = 0;
  if constexpr (TOP) {
    k = join_best<WAVES>(best, lists, counts, all, P.top);
  }
  if (lane == 0) stats[wid] = t;
  __syncthreads();
  if (wid) return;
  t = wave_join(lane < WAVES ? stats[lane] : Stat{NEG_INF, 0.0, 0.0}, c);
  if (P.parts > 1) {
    double *o = P.stats + 3 * (int64_t)blockIdx.x;
    if (lane == 0) {
      o[0] = (double)t.m;
      o[1] = t.s;
      o[2] = t.a;
    }
    if (TOP && lane < LIST) P.keys[(int64_t)blockIdx.x * LIST + lane] = k;
    return;
  }
  finish(P, n, t, k, zt, bad);
}

// The parts of a row, lane p part p's sums; of the lists, wave w joins every WAVES-th, then they
// are joined in pairs.  One wave where there are none.
template <int DT, int WAVES> __global__ __launch_bounds__(64 * WAVES) void join_kernel(LogprobsP P) {
  __shared__ Key lists[WAVES][LIST];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int64_t n = blockIdx.x;
  const int token = P.tokens[n];
  if (token == P.ignore) return;
  const float c = LOG2E / P.T;
  const bool bad = token < 0 || token >= P.V;
  Stat t = {NEG_INF, 0.0, 0.0};
  float zt = 0.f;
  if (wid == 0) {
    if (!bad) zt = load_elem<DT>(P.z + n * P.z_ld, token);
    if (lane < P.parts) {
      const double *o = P.stats + 3 * (n * P.parts + lane);
      t = Stat{(float)o[0], o[1], o[2]};
    }
    t = wave_join(t, c);
  }
  Key k = 0;
  if constexpr (WAVES > 1) {
    const Key *keys = P.keys + n * P.parts * LIST;
    for (int p = wid; p < P.parts; p += WAVES) {
      const Key other = lane >= LIST ? keys[p * LIST + lane - LIST] : k;
      k = p == wid ? __shfl(other, lane + LIST) : merge_lists(other);
    }
    k = join_lists<WAVES>(k, lists);
  }
  if (wid == 0) finish(P, n, t, k, zt, bad);
}

template <int DT> void launch(const LogprobsP &P, int waves, int64_t n, hipStream_t st) {
  const dim3 grid((unsigned)(n * P.parts)), block(64 * waves);
  if (waves == 4) {
    if (P.top) hipLaunchKernelGGL((logprobs_kernel<DT, 4, true>), grid, block, 0, st, P);
    else hipLaunchKernelGGL((logprobs_kernel<DT, 4, false>), grid, block, 0, st, P);
  } else {
    if (P.top) hipLaunchKernelGGL((logprobs_kernel<DT, 16, true>), grid, block, 0, st, P);
    else hipLaunchKernelGGL((logprobs_kernel<DT, 16, false>), grid, block, 0, st, P);
  }
  if (P.parts > 1) {
    if (P.top) hipLaunchKernelGGL((join_kernel<DT, 16>), dim3((unsigned)n), dim3(1024), 0, st, P);
    else hipLaunchKernelGGL((join_kernel<DT, 1>), dim3((unsigned)n), dim3(64), 0, st, P);
  }
}

// ------------------------------------------------------------------- gradient
struct GradP {
  const char *z;
  int64_t z_ld;                          // bytes
  const int32_t *tokens;
  const float *norm, *entropy, *g, *h;
  char *grad;
  int64_t g_ld;                          // bytes
  int32_t N, V, tiles, ignore;           // N: of all rows, between the norm's two parts
  float T;
};

constexpr float LEAST = 160.f;           // 2^-LEAST and less are 0 in fp32

// One tile of a row: 256 threads, VECS vectors each.  A thread has read its entries before
// it writes them, so the gradient may lie where the logits do.
template <int DT, int GT> __global__ __launch_bounds__(256) void grad_kernel(GradP P) {
  constexpr int E = Fmt<DT>::E, W = Fmt<DT>::W, GE = Fmt<GT>::E;
  const int64_t n = blockIdx.x / P.tiles;
  const int64_t at = (int64_t)(blockIdx.x - n * P.tiles) * (256 * VECS * W) + (int64_t)threadIdx.x * W;
  const int token = P.tokens[n];
  const float m = P.norm[n], ls = P.norm[P.N + n], inv = 1.f / P.T, c = LOG2E / P.T;
  const bool used = token != P.ignore && token >= 0 && token < P.V && fabsf(m) < __builtin_inff() && fabsf(ls) < __builtin_inff();
  float g = 0.f, h = 0.f, hs = 0.f;
  if (used) {
    g = P.g[n];
    if (P.h) {
      h = P.h[n];
      hs = h * P.entropy[n];
    }
  }
  u32x4 r[VECS];
  if (used) {
    load_step<DT, 4>(P.z + n * P.z_ld, at, P.V, r);
  }
  // 1 / T is in the factors, unless they would leave fp32 (T below 1e-34, say, where entries of
  // probability 0 would be 0 times infinity): then it comes to the results.
  const bool fits = (fabsf(g) + fabsf(hs) + LEAST * fabsf(h)) * inv < __builtin_inff();
  const float before = fits ? inv : 1.f, behind = fits ? 1.f : inv;
  const float k0 = -(g + hs) * before, k1 = -h * (float)LN2 * before, l2 = ls * LOG2E;
  char *o = P.grad + n * P.g_ld;
#pragma unroll
  for (int s = 0; s < VECS; ++s) {
    const int64_t e = at + (int64_t)s * (256 * W);
    float v[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      v[w] = 0.f;
      if (used) {
        const float t = __builtin_fmaxf(fmaf(unpack<DT>(r[s], w) - m, c, -l2), -LEAST);   // log2 p
        v[w] = __builtin_amdgcn_exp2f(t) * fmaf(t, k1, k0);
      }
    }
    if (used && token >= e && token < e + W) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (token == e + w) v[w] += g * before;
    }
#pragma unroll
    for (int w = 0; w < W; ++w) v[w] *= behind;
    if (e + W <= P.V) {
      if constexpr (GT == SV_BF16) {
        uint32_t u[W / 2];
#pragma unroll
        for (int q = 0; q < W / 2; ++q)
          u[q] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * q]) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * q + 1]) << 16;
        if constexpr (W == 8) {
          __builtin_nontemporal_store(u32x4{u[0], u[1], u[2], u[3]}, (u32x4_any *)(o + e * GE));
        } else {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          typedef u32x2 u32x2_any __attribute__((aligned(2)));
          __builtin_nontemporal_store(u32x2{u[0], u[1]}, (u32x2_any *)(o + e * GE));
        }
      } else {
#pragma unroll
        for (int q = 0; q < W / 4; ++q)
          __builtin_nontemporal_store(u32x4{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                            __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])},
                                      (u32x4_any *)(o + e * GE) + q);
      }
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (e + w < P.V) {
          if constexpr (GT == SV_BF16) ((__bf16 *)o)[e + w] = (__bf16)v[w];
          else ((float *)o)[e + w] = v[w];
        }
    }
  }
}

template <int DT, int GT> void launch_grad(const GradP &P, int64_t n, hipStream_t st) {
  hipLaunchKernelGGL((grad_kernel<DT, GT>), dim3((unsigned)(n * P.tiles)), dim3(256), 0, st, P);
}

}  // namespace

extern "C" size_t sv_logprobs_workspace_bytes(const sv_logprobs_shape_t *s) {
  if (!s || !sv_logprobs_host::temperature_ok(s->temperature) || !sv_logprobs_host::shape_ok(s)) return 0;
  return sv_logprobs_host::plan_for(s).total;
}

extern "C" int sv_logprobs(const sv_logprobs_shape_t *shape, const void *logits, const int32_t *tokens, float *logp,
                           float *entropy, float *lse, float *norm, int32_t *status, float *top_logp, int32_t *top_idx,
                           void *workspace, size_t workspace_bytes, void *stream) {
  bool nothing;
  const int rc = sv_logprobs_host::check(shape, logits, tokens, logp, top_logp, top_idx, workspace, workspace_bytes,
                                         &nothing);
  if (rc != SV_OK || nothing) return rc;
  const sv_logprobs_shape_t &s = *shape;
  const sv_logprobs_host::Plan L = sv_logprobs_host::plan_for(&s);
  LogprobsP P = {};
  P.z = (const char *)logits;
  P.z_ld = (s.row_stride ? s.row_stride : s.V) * sv_logprobs_host::esize(s.dtype);
  P.tokens = tokens;
  P.logp = logp;
  P.entropy = entropy;
  P.lse = lse;
  P.norm = norm;
  P.status = status;
  P.top_logp = top_logp;
  P.top_idx = top_idx;
  P.N = s.N;
  P.V = s.V;
  P.top = s.top;
  P.ignore = s.ignore_index;
  P.parts = L.parts;
  P.batch = L.batch;
  P.batches = L.batches;
  P.T = s.temperature;
  P.stats = (double *)((char *)workspace + L.stats);
  P.keys = (Key *)((char *)workspace + L.keys);
  if (s.dtype == SV_BF16) launch<SV_BF16>(P, L.waves, s.N, (hipStream_t)stream);
  else launch<SV_F32>(P, L.waves, s.N, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int sv_logprobs_grad(const sv_logprobs_grad_shape_t *shape, const void *logits, const int32_t *tokens,
                                const float *norm, const float *entropy, const float *grad_logp,
                                const float *grad_entropy, void *grad, void *stream) {
  bool nothing;
  const int rc = sv_logprobs_host::check_grad(shape, logits, tokens, norm, entropy, grad_logp, grad_entropy, grad,
                                              &nothing);
  if (rc != SV_OK || nothing) return rc;
  const sv_logprobs_grad_shape_t &s = *shape;
  const hipStream_t st = (hipStream_t)stream;
  const int e = sv_logprobs_host::esize(s.dtype), ge = sv_logprobs_host::esize(s.grad_dtype);
  GradP P = {};
  P.z_ld = (s.row_stride ? s.row_stride : s.V) * e;
  P.g_ld = (s.grad_stride ? s.grad_stride : s.V) * ge;
  P.N = s.N;
  P.V = s.V;
  P.tiles = (int32_t)cdiv(s.V, 256 * VECS * (16 / e));
  P.ignore = s.ignore_index;
  P.T = s.temperature;
  const int64_t most = sv_head_host::max_groups(256) / P.tiles;   // rows of a launch
  for (int64_t n = 0; n < s.N; n += most) {
    const int64_t rows = s.N - n < most ? s.N - n : most;
    P.z = (const char *)logits + n * P.z_ld;
    P.tokens = tokens + n;
    P.norm = norm + n;
    P.entropy = entropy ? entropy + n : nullptr;
    P.g = grad_logp + n;
    P.h = grad_entropy ? grad_entropy + n : nullptr;
    P.grad = (char *)grad + n * P.g_ld;
    if (s.dtype == SV_BF16) {
      if (s.grad_dtype == SV_BF16) launch_grad<SV_BF16, SV_BF16>(P, rows, st);
      else launch_grad<SV_BF16, SV_F32>(P, rows, st);
    } else {
      if (s.grad_dtype == SV_BF16) launch_grad<SV_F32, SV_BF16>(P, rows, st);
      else launch_grad<SV_F32, SV_F32>(P, rows, st);
    }
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
