// Softmax + top-k routing and its backward (Aurora page, section 3.1,
// Algorithm 1 stage 1: probs = Softmax(logits); weights, indices = TopK(probs),
// with the top-k probabilities renormalised over the selection by default).
//
// One wavefront owns one token: lane l holds logits l, l+64, l+128, ... of the
// token's row (coalesced 256-byte loads), and each of the k rounds is a
// lane-local arg-max followed by a 6-step butterfly over the wave.  The order
// is (logit descending, expert index ascending), so equal logits - including
// +0.0 against -0.0 - go to the lower expert.  The whole pass reads T*E*4
// bytes and writes T*k*8; it is bound by HBM.
#include "internal.h"
#include "route.h"

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

// MAXV = ceil(E / 64): lane l holds experts l, l + 64, ... (absent ones as
// -infinity).  Each wave selects for TPW consecutive tokens, with the loads
// of all their rows issued first, so that a wave keeps TPW rows in flight
// while it works through the selections.
template <int MAXV, bool GROUPED, int TPW>
__global__ void __launch_bounds__(256) topk_route_kernel(const float* __restrict__ logits, int T, int E,
                                                         int k, int renorm, int G,
                                                         int32_t* __restrict__ idx_out,
                                                         float* __restrict__ w_out) {
  __shared__ int32_t s_idx[4][64];
  __shared__ float s_val[4][64];
  const int lane = threadIdx.x & 63;
  const int wv = threadIdx.x >> 6;
  const int t0 = (blockIdx.x * 4 + wv) * TPW;
  if (t0 >= T) return;
  float v[TPW][MAXV];
  const bool full = E == MAXV * 64;  // (uniform) every lane holds MAXV experts: no mask
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const int t = min(t0 + u, T - 1);  // (a token past T re-reads the last row, unused)
    const float* row = logits + (int64_t)t * E;
    if (full) {
#pragma unroll
      for (int i = 0; i < MAXV; ++i) v[u][i] = row[i * 64 + lane];
    } else {
#pragma unroll
      for (int i = 0; i < MAXV; ++i) {
        const int e = i * 64 + lane;
        v[u][i] = e < E ? row[e] : -INFINITY;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < TPW; ++u) {
    const int t = t0 + u;
    if (t >= T) break;
    if (GROUPED)
      topk_rounds<MAXV, GROUPED>(v[u], lane, t, E, k, renorm, G, idx_out, w_out);
    else
      topk_token<MAXV>(v[u], lane, t, E, k, renorm, idx_out, w_out, s_idx[wv], s_val[wv]);
  }
}

// dlogits, one wave per token.  renorm: dL_m = w_m (dw_m - <w, dw>) on the
// selected experts (local or not), 0 elsewhere.  raw softmax: dL_e = p_e (g_e
// - <w, dw>) with g_e = dw_j at e = idx_j.  Lane j (< k) holds slot j; <w, dw>
// is a butterfly sum over the wave.  The k values are scattered into a
// zeroed LDS copy of the token's row at their experts (the experts of a
// token are distinct), which the lanes then read back in the order they
// store the row: expert e is element e/64 of lane e%64.  (A wave's LDS
// operations complete in order, so the zeroing lands before the scatter.)
template <int MAXV>
__global__ void __launch_bounds__(256) route_bwd_kernel(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ idx,
                                                        const float* __restrict__ w,
                                                        const float* __restrict__ dw, int T, int E, int k,
                                                        int renorm, float* __restrict__ dlogits) {
  __shared__ float s_g[4][MAXV * 64];
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  float* gs = s_g[threadIdx.x >> 6];
  int my_i = 0;
  float my_w = 0.f, my_dw = 0.f;
  if (lane < k) {
    my_i = min(max(idx[(int64_t)t * k + lane], 0), E - 1);  // (clamped: no write outside the row)
    my_w = w[(int64_t)t * k + lane];
    my_dw = dw[(int64_t)t * k + lane];
  }
  const float s = wave_sum(my_w * my_dw);  // <w, dw>
#pragma unroll
  for (int i = 0; i < MAXV; ++i) gs[i * 64 + lane] = 0.f;
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  if (lane < k) gs[my_i] = renorm ? my_w * (my_dw - s) : my_dw;
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  float g[MAXV];
#pragma unroll
  for (int i = 0; i < MAXV; ++i) g[i] = gs[i * 64 + lane];
  float* out = dlogits + (int64_t)t * E;
  if (renorm) {
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int e = i * 64 + lane;
      if (e < E) out[e] = g[i];
    }
  } else {
    const float* row = logits + (int64_t)t * E;
    float v[MAXV];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int e = i * 64 + lane;
      v[i] = e < E ? row[e] : -INFINITY;
      mx = fmaxf(mx, v[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
      if (i * 64 + lane < E) z += expf(v[i] - mx);
    z = wave_sum(z);
#pragma unroll
    for (int i = 0; i < MAXV; ++i) {
      const int e = i * 64 + lane;
      if (e < E) out[e] = expf(v[i] - mx) / z * (g[i] - s);
    }
  }
}

// dlogits with renormalised weights, two tokens per wave: lanes 0-31 take
// token 2w and lanes 32-63 token 2w+1 (k <= 32), each half summing its own
// <w, dw> (the same additions as wave_sum, whose first step over the upper
// half's zeros is exact).  Both rows are zeroed in LDS, the selections
// scattered into them, and the two rows - contiguous in dlogits - written as
// 16-byte vectors (E a multiple of 8: no vector straddles two rows, and row
// 2w starts 16-byte aligned).  E2: 2 E rounded up to 256 floats (LDS per wave).
template <int E2>
__global__ void __launch_bounds__(256) route_bwd_renorm2_kernel(const int32_t* __restrict__ idx,
                                                                const float* __restrict__ w,
                                                                const float* __restrict__ dw, int T, int E, int k,
                                                                float* __restrict__ dlogits) {
  __shared__ __attribute__((aligned(16))) float s_g[4][E2];
  const int lane = threadIdx.x & 63, l = lane & 31, half = lane >> 5;
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 2;
  if (t0 >= T) return;
  const int t = t0 + half;
  float* gs = s_g[threadIdx.x >> 6];
  const bool mine = l < k && t < T;
  int my_i = 0;
  float my_w = 0.f, my_dw = 0.f;
  if (mine) {
    my_i = min(max(idx[(int64_t)t * k + l], 0), E - 1);  // (clamped: no write outside the row)
    my_w = w[(int64_t)t * k + l];
    my_dw = dw[(int64_t)t * k + l];
  }
  float s = my_w * my_dw;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);  // within each half
  const int n4 = E >> 1;  // 16-byte vectors in the two rows
  float4* g4 = reinterpret_cast<float4*>(gs);
#pragma unroll
  for (int q = lane; q < E2 / 4; q += 64)
    if (q < n4) g4[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  if (mine) gs[half * E + my_i] = my_w * (my_dw - s);
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  const int nv = (t0 + 1 < T) ? n4 : n4 >> 1;  // the second row only if token 2w+1 exists
  float4* out = reinterpret_cast<float4*>(dlogits + (int64_t)t0 * E);
#pragma unroll
  for (int q = lane; q < E2 / 4; q += 64)
    if (q < nv) out[q] = g4[q];
}

// One instantiation per number of 64-wide slices of a logit row (1 .. 16 for
// E <= 1024), so no slice is carried for nothing.
template <int NV, bool GROUPED>
static void route_nv(const moe_desc& d, int nv, const float* logits, int G, int32_t* idx, float* w,
                     hipStream_t s) {
  if constexpr (NV <= 16) {
    if (nv > NV) return route_nv<NV + 1, GROUPED>(d, nv, logits, G, idx, w, s);
    constexpr int TPW = 1;  // tokens per wave (2 measured no faster: the selection, not the loads, is the cost)
    topk_route_kernel<NV, GROUPED, TPW><<<(d.T + 4 * TPW - 1) / (4 * TPW), 256, 0, s>>>(logits, d.T, d.E, d.k,
                                                                                      d.renormalize, G, idx, w);
  }
}

template <bool GROUPED>
static void route_dispatch(const moe_desc& d, const float* logits, int G, int32_t* idx, float* w, hipStream_t s) {
  route_nv<1, GROUPED>(d, (d.E + 63) / 64, logits, G, idx, w, s);
}

template <int NV>
static void route_bwd_nv(const moe_desc& d, int nv, const float* logits, const int32_t* idx, const float* w,
                         const float* dw, float* dlogits, hipStream_t s) {
  if constexpr (NV <= 16) {
    if (nv > NV) return route_bwd_nv<NV + 1>(d, nv, logits, idx, w, dw, dlogits, s);
    if (d.renormalize) {  // two tokens per wave, E <= 64 NV
      constexpr int E2 = (2 * 64 * NV + 255) / 256 * 256;
      route_bwd_renorm2_kernel<E2><<<(d.T + 7) / 8, 256, 0, s>>>(idx, w, dw, d.T, d.E, d.k, dlogits);
      return;
    }
    // one token per wave (4 per wave measured slower: 0.050 against 0.041 ms at T = 65536, E = 384)
    route_bwd_kernel<NV><<<(d.T + 3) / 4, 256, 0, s>>>(logits, idx, w, dw, d.T, d.E, d.k, d.renormalize,
                                                          dlogits);
  }
}

hipError_t launch_route(const moe_desc& d, const float* logits, int n_groups, int32_t* idx, float* w,
                        hipStream_t s) {
  if (n_groups > 1) route_dispatch<true>(d, logits, n_groups, idx, w, s);
  else route_dispatch<false>(d, logits, 1, idx, w, s);
  return hipGetLastError();
}

hipError_t launch_route_bwd(const moe_desc& d, const float* logits, const int32_t* idx, const float* w,
                            const float* dw, float* dlogits, hipStream_t s) {
  route_bwd_nv<1>(d, (d.E + 63) / 64, logits, idx, w, dw, dlogits, s);
  return hipGetLastError();
}

}  // namespace moe
