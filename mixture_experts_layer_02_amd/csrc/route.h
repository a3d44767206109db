// The selection of one token by one wave: softmax + top-k, plain and
// group-limited (route.hip's kernels and the decode step's).
#pragma once

#include "common.h"

namespace moe {

// Group-limited selection (Domyn page, section "Group-limited expert
// routing"): with G > 1 groups of Eg = E/G consecutive experts, each group
// may give at most k/G experts.  The rounds still take the best remaining
// eligible expert, and once a group has given its quota its other experts
// leave the race, so the k picks are the union of every group's k/G best, in
// descending order (the eligible set only shrinks).  Lane g counts group g's
// picks.
//
// k rounds of a lane-local arg-max and a wave butterfly over the wave's
// token (v: the lane's logits, element i = expert i*64 + lane); writes the
// token's k selections and weights.
template <int MAXV, bool GROUPED>
__device__ __forceinline__ void topk_rounds(const float (&v)[MAXV], int lane, int t, int E, int k, int renorm,
                                            int G, int32_t* __restrict__ idx_out, float* __restrict__ w_out) {
  uint32_t taken = 0;  // bit i: element i is selected already or absent
#pragma unroll
  for (int i = 0; i < MAXV; ++i)
    if (i * 64 + lane >= E) taken |= 1u << i;
  float my_v = 0.f, v0 = 0.f;
  int my_i = 0;
  const int Eg = GROUPED ? E / G : E, kg = GROUPED ? k / G : k;
  int group_picks = 0;  // lane g: experts taken from group g so far
  for (int j = 0; j < k; ++j) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      if (!((taken >> i) & 1u) && (bi == 0x7fffffff || v[i] > bv)) {
        bv = v[i];
        bi = i * 64 + lane;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float ov = __shfl_xor(bv, o, 64);
      const int oi = __shfl_xor(bi, o, 64);
      const bool better = (oi != 0x7fffffff) && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi));
      if (better) {
        bv = ov;
        bi = oi;
      }
    }
    if ((bi & 63) == lane) taken |= 1u << (bi >> 6);
    if (GROUPED) {
      const int g = bi / Eg;
      if (lane == g) ++group_picks;
      if (__shfl(group_picks, g, 64) == kg) {  // the group is full: its other experts leave
#pragma unroll
        for (int i = 0; i < MAXV; ++i)
          if ((i * 64 + lane) / Eg == g) taken |= 1u << i;
      }
    }
    if (lane == j) {
      my_v = bv;
      my_i = bi;
    }
    if (j == 0) v0 = bv;
  }
  float w;
  if (renorm) {
    const float ex = lane < k ? expf(my_v - v0) : 0.f;
    w = ex / wave_sum(ex);
  } else {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
      if (i * 64 + lane < E) s += expf(v[i] - v0);
    s = wave_sum(s);
    w = expf(my_v - v0) / s;
  }
  if (lane < k) {
    idx_out[(int64_t)t * k + lane] = my_i;
    w_out[(int64_t)t * k + lane] = w;
  }
}

// Order-preserving unsigned key of a float (larger float, larger key), with
// -0.0 made equal to +0.0; 0 is below every finite float's key and marks an
// absent element.  key_float inverts it (+0.0 for the key of zero).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0.0 + 0.0 = +0.0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// The selection of one token t by one wave: v holds the token's logits,
// element i of lane l being expert i*64 + l (absent experts -infinity);
// s_idx / s_val are the wave's 64-entry LDS area.
template <int MAXV>
__device__ __forceinline__ void topk_token(const float (&v)[MAXV], int lane, int t, int E, int k, int renorm,
                                           int32_t* __restrict__ idx_out, float* __restrict__ w_out,
                                           int32_t* s_idx, float* s_val) {
  // Threshold selection.  theta = the k-th largest of the lanes' maximum keys
  // (a binary search over the key bits, counting lanes with ballots), or a
  // key below it: at least k elements have key >= theta, so every one of the
  // k selections does, and the candidates (key >= theta) are usually few.
  // They are compacted through LDS, and a candidate's slot is the number of
  // candidates that come before it in the order (logit descending, expert
  // ascending).  With more than 64 candidates (heavy ties) the wave takes
  // the k rounds instead.  Only the lane maxima need keys: theta is the key
  // of a float, so key >= theta is the float comparison v >= key_float(theta),
  // under which -0.0 and +0.0 are equal too.
  float vmax = v[0];
#pragma unroll
  for (int i = 1; i < MAXV; ++i) vmax = fmaxf(vmax, v[i]);
  const uint32_t kmax = lane < E ? order_key(vmax) : 0u;  // a lane holds an expert iff lane < E
  // The search runs over the top 16 key bits only: theta is then the k-th
  // largest lane maximum with its low 16 bits cleared, still at or below it,
  // so the candidates still hold every selection; values within 2^-7 of it
  // add the odd extra candidate.  (A theta below the key of -infinity would
  // name a NaN; it is raised to that key, and every element is a candidate.)
  // (uicmp: the lanes' unsigned kmax >= c as a wave mask in one compare,
  // without materialising the predicate first as a ballot does)
  uint32_t theta = 0;
  for (int b = 31; b >= 16; --b) {
    const uint32_t c = theta | (1u << b);
    if ((int)__popcll(__builtin_amdgcn_uicmp(kmax, c, 35 /* unsigned >= */)) >= k) theta = c;
  }
  if (theta < 0x00800000u) theta = 0x007FFFFFu;
  const float thf = key_float(theta);
  uint64_t m[MAXV];
  int cnt = 0;
#pragma unroll
  for (int i = 0; i < MAXV; ++i) {
    m[i] = __ballot(v[i] >= thf);  // absent experts are -infinity, below every finite theta
    cnt += (int)__popcll(m[i]);
  }
  if (cnt > 64) {  // uniform
    topk_rounds<MAXV, false>(v, lane, t, E, k, renorm, 1, idx_out, w_out);
    return;
  }
  int base = 0;
#pragma unroll
  for (int i = 0; i < MAXV; ++i) {
    if (v[i] >= thf) {  // (this lane's bit of m[i]); pos = base + the set bits of m[i] below the lane
      const int pos = base + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m[i] >> 32),
                                                             __builtin_amdgcn_mbcnt_lo((uint32_t)m[i], 0u));
      s_idx[pos] = i * 64 + lane;
      s_val[pos] = v[i];
    }
    base += (int)__popcll(m[i]);
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  const bool cand = lane < cnt;
  const int ci = cand ? s_idx[lane] : 0x7fffffff;
  const float cv = cand ? s_val[lane] : 0.f;
  // rank = candidates before this one in (logit descending, expert
  // ascending): one unsigned compare of (key, ~expert) pairs
  const uint32_t khi = order_key(cv), klo = ~(uint32_t)ci;
  const uint64_t ck = ((uint64_t)khi << 32) | klo;
  int rank = 0;
  for (int j = 0; j < cnt; ++j) {
    const uint64_t kj = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)khi, j) << 32) |
                        (uint32_t)__builtin_amdgcn_readlane((int)klo, j);
    rank += kj > ck ? 1 : 0;
  }
  const bool sel = cand && rank < k;
  // the largest selected logit (slot 0)
  const uint64_t top = __ballot(cand && rank == 0);
  const float v0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cv), (int)__builtin_ctzll(top)));
  // Weights with the hardware exp2 and reciprocal (a few ulp; their
  // exponents x <= 0).
  float w;
  if (renorm) {
    const float ex = sel ? __expf(cv - v0) : 0.f;
    w = ex * __builtin_amdgcn_rcpf(wave_sum(ex));
  } else {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
      if (i * 64 + lane < E) s += __expf(v[i] - v0);
    s = wave_sum(s);
    w = __expf(cv - v0) * __builtin_amdgcn_rcpf(s);
  }
  if (sel) {
    idx_out[(int64_t)t * k + rank] = ci;
    w_out[(int64_t)t * k + rank] = w;
  }
}

}  // namespace moe
