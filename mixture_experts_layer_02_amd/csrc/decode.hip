// The whole expert layer for a few tokens (T <= 64) in two kernels: the router
// logits, then everything else.
//
// At these sizes the layer streams the weights of the experts that the tokens
// take, each byte once, and is bound by HBM; the rest is latency.  The second
// kernel therefore has one workgroup per CU, whose waves copy weights from
// start to end (stream.h): every workgroup selects for all tokens by itself (a
// few hundred logits each, cheaper than a kernel or a hand-over; of more tokens
// than it has waves, a workgroup selects for one and flags it), then
//   phase 1: (expert, 8 channels of f or more) items: gate and up rows over all
//            of d, h = silu(G) U to memory as bf16 (as in the layer's other forms,
//            and what the matrix cores take: y is then 0.0024 of its rms from the
//            exact sums, with its own rounding alone 0.0017),
//   phase 2: (8 or 24 channels of d) items: for every expert hit, its W2 rows
//            over all of f, times the routing weights, summed over the experts
//            in LDS, so that y is written once and no atomics change its order.
// Between the phases all of h has to be there.  Each workgroup raises a flag
// when its phase-1 items are done and waits for all flags (they take 3 to 4 us
// from the last one on; looked at faster, all 256 in one go or one counter in
// their place, the looking holds up the raising: 7 and 12 us); the W2 copies of its
// first phase-2 items are in flight meanwhile.
//
// The wait needs no workgroup that is not running yet: a workgroup's items
// belong to a number that it takes from a counter when it starts, and one that
// has waited for a while takes further numbers, those of workgroups that have
// not started, and does their items first; a workgroup that gets a number past
// the last one has nothing to do.  So kernels that hold compute units, another
// decode step among them, cannot stop it.
//
// W waves stream; one more serves: it adds up the waves' partial sums of phase
// 1 and stores h while the others are at the next item.
#include <algorithm>

#include "internal.h"
#include "route.h"
#include "stream.h"

namespace moe {

namespace {

using dma::lds_barrier;

constexpr int MAX_T = MOE_DECODE_MAX_T, MAX_K = 32, MAX_E = 1024;
// sync[0]: the counter of workgroups; sync[SYNC_TOKENS + t]: token t's selection is
// there; sync[SYNC_FLAGS + i]: number i's phase 1 is done.
constexpr int SYNC_TOKENS = 64, SYNC_FLAGS = SYNC_TOKENS + MAX_T;

// ---------------------------------------------------------------------------
// Router logits
// ---------------------------------------------------------------------------

// Partial sums part[ks][t][e] of x Wr^T: a workgroup has 16 experts and a
// gridDim.y-th of d, each of its 16 waves a sixteenth of that; 16 CT tokens.  Clears the second
// kernel's counters and flags.
template <int CT>
__global__ void __launch_bounds__(1024) decode_router_kernel(const uint16_t* __restrict__ x,
                                                            const uint16_t* __restrict__ wr, int T, int d, int E,
                                                            float* __restrict__ part, uint32_t* __restrict__ sync,
                                                            int nsync) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  constexpr int W = 16;
  __shared__ float red[W][CT * 16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < nsync; i += 64 * W) sync[i] = 0;
  if (!wr) return;  // (the routing is given)
  const int steps = d / 32, parts = gridDim.y * W, me = blockIdx.y * W + wave;
  const int s0 = steps * me / parts, s1 = steps * (me + 1) / parts;
  const uint16_t* a = wr + (int64_t)min((int)blockIdx.x * 16 + r, E - 1) * d + q * 8;
  const uint16_t* b[CT];
  f32x4_t acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    b[c] = x + (int64_t)min(c * 16 + r, T - 1) * d + q * 8;
    acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  constexpr int U = CT == 1 ? 4 : 2;  // steps whose loads are in flight together
  for (int s = s0; s < s1; s += U) {
    bf16x8 fa[U], fb[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(s + u, s1 - 1) * 32;
      fa[u] = *reinterpret_cast<const bf16x8*>(a + at);
#pragma unroll
      for (int c = 0; c < CT; ++c) fb[u][c] = *reinterpret_cast<const bf16x8*>(b[c] + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[u], fb[u][c], acc[c], 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][c * 16 + r][4 * q + i] = acc[c][i];
  __syncthreads();
  for (int i = tid; i < CT * 256; i += 64 * W) {
    const int t = i >> 4, e = (int)blockIdx.x * 16 + (i & 15);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[w][t][i & 15];
    if (t < T && e < E) part[((int64_t)blockIdx.y * T + t) * E + e] = sum;
  }
}

// ---------------------------------------------------------------------------
// The rest
// ---------------------------------------------------------------------------

struct DecodeParams {
  const uint16_t* x;
  const uint8_t *w1, *w3, *w2;
  const float *s1, *s3, *s2;
  const float* part;  // logits' partial sums; NULL: idx and w are given
  const float* bias;
  int32_t* idx;
  float* w;
  uint16_t* h;  // [T k][f], by slot
  uint16_t* y;
  uint32_t* sync;
  int T, d, f, E, k, e0, NL, renorm, n_groups, ks;
};

constexpr __host__ __device__ int align128(int n) { return (n + 127) / 128 * 128; }

// The tokens that one pass over an expert's rows serves.
struct alignas(8) Block {
  uint16_t e, n;   // local expert; tokens (<= RB)
  uint16_t pos;    // their place in the list of rows
  uint8_t off, nb; // which of the expert's blocks it is, and of how many
};

// The largest of v over each aligned group of L lanes (a power of two), in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int L) {
  if (L >= 2) v = dpp_max<0xB1>(v);    // quad_perm:[1,0,3,2]
  if (L >= 4) v = dpp_max<0x4E>(v);    // quad_perm:[2,3,0,1]
  if (L >= 8) v = dpp_max<0x141>(v);   // row_half_mirror
  if (L >= 16) v = dpp_max<0x140>(v);  // row_mirror
  if (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(s[0], s[1]);
  }
  if (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(s[0], s[1]);
  }
  return v;
}

// The selection of token t by one wave, as moe_route and moe_route_grouped
// define it, to idx and w ([k], LDS).  keys: the wave's E words of LDS; pick: 2 k
// words.  A group of experts belongs to L lanes, which hold its experts l, l + L,
// ..; every group's best k / n_groups are taken one after the other, the groups
// side by side: a lane knows its best, the group's is found over the lanes, and
// its lane looks through its experts again.  Short code rather than few steps: it
// runs once per launch, from a cold instruction cache (unrolled, with a token's
// logits in registers, the kernel was 128 KB long, and 12 tokens in 4 groups took
// 20 us).
__device__ __forceinline__ void route_token(const DecodeParams& p, int t, int lane, uint32_t* keys, uint32_t* pick,
                                            int32_t* idx, float* w) {
  // (the loads of four experts a lane together: one after the other they took 1.5 us each)
  for (int e0 = lane; e0 < p.E; e0 += 256) {
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = min(e0 + 64 * u, p.E - 1);
      const float* row = p.part + (int64_t)t * p.E + e;
      const int64_t ld = p.ks == 1 ? 0 : (int64_t)p.T * p.E;
      const float b = p.bias ? p.bias[e] : 0.f;
      v[u] = p.ks == 1 ? b + row[0] : b + ((row[0] + row[ld]) + (row[2 * ld] + row[3 * ld]));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e0 + 64 * u < p.E) keys[e0 + 64 * u] = max(order_key(v[u]), 1u);  // 0: taken
  }
  const int Eg = p.E / p.n_groups, kg = p.k / p.n_groups;
  const int L = p.n_groups == 1 ? 64 : 64 >> (32 - __builtin_clz(p.n_groups - 1));
  const int g = lane / L, l = lane % L;
  const bool has = g < p.n_groups;
  uint32_t best = 0, at = 0;
  auto look = [&]() {
    best = 0;
    for (int e = l; e < Eg; e += L) {
      const uint32_t v = keys[g * Eg + e];
      if (v > best) best = v, at = e;
    }
  };
  if (has) look();
  for (int r = 0; r < kg; ++r) {
    const uint32_t top = lanes_max(best, L);
    const uint32_t e = ~lanes_max(best == top ? ~at : 0u, L);  // the lowest of equals
    if (has && best == top && at == e) {
      pick[g * kg + r] = top;
      pick[p.k + g * kg + r] = g * Eg + e;
      keys[g * Eg + e] = 0;
      look();
    }
  }
  __builtin_amdgcn_wave_barrier();
  const uint32_t my_key = lane < p.k ? pick[lane] : 0, my_i = lane < p.k ? pick[p.k + lane] : 0;
  // Slots in falling order: pick j's is the number of picks before it.
  int rank = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t kj = (uint32_t)__builtin_amdgcn_readlane((int)my_key, j);
    const uint32_t ij = (uint32_t)__builtin_amdgcn_readlane((int)my_i, j);
    rank += kj > my_key || (kj == my_key && ij < my_i);
  }
  const float v0 = key_float(lanes_max(my_key, 64));
  const float ex = lane < p.k ? expf(key_float(my_key) - v0) : 0.f;
  float sum = ex;
  if (!p.renorm)
    for (int e = lane; e < p.E; e += 64)
      if (keys[e]) sum += expf(key_float(keys[e]) - v0);
  sum = wave_sum(sum);
  if (lane < p.k) {
    idx[rank] = (int)my_i;
    w[rank] = ex / sum;
  }
}

// GRP 0: bf16 weights.  TMAX tokens at most, RB of them in a pass over an expert's
// rows.  R1 rows (half gate, half up) a stage in phase 1, R2 by SUB2 pieces of 128
// bytes in phase 2; W streaming waves.  LDS holds the lists, then the rings and, before
// them, phase 1's partial sums or phase 2's sums per token.
template <int GRP, int TMAX, int RB, int R1, int R2, int SUB2, int W>
__global__ void __launch_bounds__(64 * (W + 1)) decode_kernel(DecodeParams p) {
  using namespace stream;
  using ST1 = Stage<GRP, R1, 1, true, RB>;
  using ST2 = Stage<GRP, R2, SUB2, false, RB>;
  constexpr int PRE1 = ST1::WI + ST1::SI, PRE2 = ST2::WI + ST2::SI;  // copies of a stage's weights
  constexpr int RP = R1 + 4;  // pitch of phase 1's partial sums (floats)
  constexpr int NT = 64 * (W + 1), LDS = 159 * 1024;
  // (stages at most; as many as there is room for with the rows that they have)
  constexpr int MOST1 = LDS / W / ST1::bytes(1) < 8 ? LDS / W / ST1::bytes(1) : 8;
  constexpr int MOST2 = LDS / W / ST2::bytes(1) < 8 ? LDS / W / ST2::bytes(1) : 8;
  constexpr int ROWS = TMAX * MAX_K, EXPERTS = ROWS < MAX_E ? ROWS : MAX_E;
  // (an expert of n rows has at most 1 + (n - 1) / RB blocks)
  constexpr int BLOCKS = EXPERTS + (TMAX <= RB ? 0 : (ROWS - EXPERTS) / RB);
  // Scratch of the selection, over the ring before it starts.
  constexpr int O_IDX = 0, O_W = O_IDX + ROWS * 4, O_MASK = O_W + ROWS * 4, O_BASE = O_MASK + MAX_E * 8,
                O_KEY = O_BASE + MAX_E * 2, KEYS = MAX_E + 2 * MAX_K, SCRATCH = O_KEY + (W + 1) * KEYS * 4;
  // With the most rows and tokens there is room for a stage of each wave.
  constexpr int LISTS = align128(BLOCKS * 8 + ROWS * 8);
  static_assert(LISTS + SCRATCH <= LDS, "scratch");
  static_assert((LDS - LISTS - align128(2 * W * RB * RP * 4)) / W / 128 * 128 >= ST1::BYTES, "a stage");
  static_assert((LDS - LISTS - align128(2 * W * RB * RP * 4)) / W / 128 * 128 >= ST2::BYTES, "a stage");
  static_assert((LDS - LISTS - align128(W * TMAX * R2 * 4)) / W / 128 * 128 >= ST2::BYTES, "a stage");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
  __shared__ uint16_t s_more[256];  // numbers taken over
  __shared__ int s_vid, s_nblk, s_rows, s_cmd;
  __shared__ uint64_t s_todo;

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = gridDim.x, slots = p.T * p.k;
  // The lists come first in LDS; the rest is phase 1's sums or phase 2's, and the
  // rings.  Above 16 tokens they are sized for this call, not for the most that there
  // may be, which left one stage a wave in phase 2 (4 bits, in turn on one card: the share's
  // 64 tokens 285 -> 280 us, 24 tokens of 96 experts 348 -> 331, 64 of them 456 -> 461;
  // for fewer tokens the sizes that are known beforehand are 0.5 us better).
  constexpr bool SIZED = TMAX > 16;
  const int hits = min(slots, p.NL), blocks = SIZED ? hits + (slots - hits) / RB : BLOCKS, listed = SIZED ? slots : ROWS;
  Block* s_blk = reinterpret_cast<Block*>(smem);
  float* s_roww = reinterpret_cast<float*>(smem + blocks * 8);
  uint32_t* s_row = reinterpret_cast<uint32_t*>(smem + blocks * 8 + listed * 4);  // slots (low 16 bits) and tokens of the rows, by expert
  const int lists = align128(blocks * 8 + listed * 8);
  uint8_t* pool = smem + lists;

  // ---- the selection, and the rows by expert
  int32_t* l_idx = reinterpret_cast<int32_t*>(pool + O_IDX);
  float* l_w = reinterpret_cast<float*>(pool + O_W);
  unsigned long long* l_mask = reinterpret_cast<unsigned long long*>(pool + O_MASK);
  uint16_t* l_base = reinterpret_cast<uint16_t*>(pool + O_BASE);
  int number = 0;
  if (tid == 64 * W) number = (int)__hip_atomic_fetch_add(p.sync, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < p.NL; i += NT) l_mask[i] = 0;
  if (p.part) {
    // Up to a token a wave: every workgroup selects for all.  More: one workgroup
    // each, and the others wait for its flag, but not for long: if it has not
    // started, they select for themselves.
    uint32_t* keys = reinterpret_cast<uint32_t*>(pool + O_KEY) + wave * KEYS;
    const bool shared = p.T > W + 1;
    uint64_t todo = ~0ull >> (64 - p.T);  // tokens to select for here
    if (shared) {
      for (int t = blockIdx.x; t < p.T; t += G) {
        if (wave == 0) {
          route_token(p, t, lane, keys, keys + MAX_E, l_idx + t * p.k, l_w + t * p.k);
          __builtin_amdgcn_wave_barrier();
          if (lane < p.k) {
            __hip_atomic_store(p.idx + t * p.k + lane, l_idx[t * p.k + lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(p.w + t * p.k + lane, l_w[t * p.k + lane], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          }
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          if (lane == 0)
            __hip_atomic_store(p.sync + SYNC_TOKENS + t, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
      if (wave == 0) {
        const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
        for (;;) {
          const bool there = lane >= p.T || __hip_atomic_load(p.sync + SYNC_TOKENS + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          todo = ~__ballot(there);
          if (todo == 0 || __builtin_amdgcn_s_memrealtime() - t0 > 3000) break;  // 30 us
          __builtin_amdgcn_s_sleep(1);
        }
        if (lane == 0) s_todo = todo;
      }
      __syncthreads();
      todo = s_todo;
      for (int i = tid; i < slots; i += NT)
        if (!(todo >> (i / p.k) & 1)) {
          l_idx[i] = __hip_atomic_load(p.idx + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          l_w[i] = __hip_atomic_load(p.w + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
#pragma nounroll
    for (int t = wave; t < p.T; t += W + 1)
      if (todo >> t & 1) route_token(p, t, lane, keys, keys + MAX_E, l_idx + t * p.k, l_w + t * p.k);
  } else {
    for (int i = tid; i < slots; i += NT) l_idx[i] = p.idx[i], l_w[i] = p.w[i];
  }
  if (tid == 64 * W) s_vid = number;
  const bool single = TMAX <= 2 && p.T == 1;
  if (single && wave == 0) {  // one token: its local slots are the blocks, in their order
    if (!p.part && lane < p.k) l_idx[lane] = p.idx[lane], l_w[lane] = p.w[lane];  // (not left to the other waves' copies)
    __builtin_amdgcn_wave_barrier();
    const uint32_t e = lane < p.k ? (uint32_t)l_idx[lane] - (uint32_t)p.e0 : ~0u;
    float w = lane < p.k ? l_w[lane] : 0.f;
    bool first = e < (uint32_t)p.NL;
    if (!p.part)  // (a second slot with the same expert adds its weight to the first)
      for (int j = 0; j < p.k; ++j) {
        if (j < lane && l_idx[j] == l_idx[lane]) first = false;
        if (j > lane && lane < p.k && l_idx[j] == l_idx[lane]) w += l_w[j];
      }
    const uint64_t m = __ballot(first);
    if (first) {
      const int pos = __popcll(m & ((1ull << lane) - 1));
      s_blk[pos] = Block{(uint16_t)e, 1, (uint16_t)pos, 0, 1};
      s_row[pos] = (uint32_t)lane;
      s_roww[pos] = w;
    }
    if (lane == 0) s_nblk = __popcll(m), s_rows = 1;
    if (p.part && blockIdx.x == 0 && lane < p.k) p.idx[lane] = l_idx[lane], p.w[lane] = l_w[lane];
  }
  __syncthreads();
  if (p.part && !single && p.T <= W + 1 && blockIdx.x == 0)
    for (int i = tid; i < slots; i += NT) p.idx[i] = l_idx[i], p.w[i] = l_w[i];
  const int vid = __builtin_amdgcn_readfirstlane(s_vid);
  if (vid >= G) return;  // (another workgroup has done this one's items)
  if (!single) {
    for (int i = tid; i < slots; i += NT) {
      const uint32_t e = (uint32_t)l_idx[i] - (uint32_t)p.e0;
      if (e < (uint32_t)p.NL) atomicOr(&l_mask[e], 1ull << (i / p.k));
    }
    __syncthreads();
    if (wave == 0) {  // exclusive sums of the experts' rows and blocks, 64 experts at a time
      uint32_t before = 0;
      int rows = 1;
#pragma nounroll
      for (int base = 0; base < p.NL; base += 64) {
        const int e = base + lane;
        const int n = e < p.NL ? __popcll(l_mask[e]) : 0, nb = (n + RB - 1) / RB;
        const uint32_t mine = (uint32_t)n | (uint32_t)nb << 16;
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const uint32_t v = __shfl_up(inc, o, WAVE);
          if (lane >= o) inc += v;
        }
        const uint32_t ex = before + inc - mine;
        if (e < p.NL) l_base[e] = (uint16_t)ex;
        rows = max(rows, min(RB, n));
        for (int b = 0; b < nb; ++b)
          s_blk[(ex >> 16) + b] = Block{(uint16_t)e, (uint16_t)min(RB, n - b * RB), (uint16_t)((ex & 0xffff) + b * RB),
                                        (uint8_t)b, (uint8_t)nb};
        before += __shfl(inc, 63, WAVE);
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) rows = max(rows, __shfl_xor(rows, o, WAVE));
      if (lane == 0) s_nblk = (int)(before >> 16), s_rows = rows;
    }
    __syncthreads();
    for (int i = tid; i < slots; i += NT) {
      const uint32_t e = (uint32_t)l_idx[i] - (uint32_t)p.e0;
      if (e >= (uint32_t)p.NL) continue;
      const int t = i / p.k;
      // a token's second slot with the same expert adds its weight to the first
      bool first = true;
      float w = l_w[i];
      if (!p.part)
        for (int j = t * p.k; j < (t + 1) * p.k; ++j) {
          if (j < i && l_idx[j] == l_idx[i]) first = false;
          if (j > i && l_idx[j] == l_idx[i]) w += l_w[j];
        }
      if (!first) continue;
      const int pos = l_base[e] + __popcll(l_mask[e] & ((1ull << t) - 1));
      s_row[pos] = (uint32_t)i | (uint32_t)t << 16;
      s_roww[pos] = w;
    }
    __syncthreads();
  }

  // ---- items
  constexpr int PR1 = R1 / 2;
  const int nblk = __builtin_amdgcn_readfirstlane(s_nblk);
  // The rings' stages have room for the rows of the largest block: of a few rows
  // more of them fit.
  const int rows = __builtin_amdgcn_readfirstlane(s_rows);
  const int bytes1 = ST1::bytes(rows), bytes2 = ST2::bytes(rows);
  const int col = ST1::column(lane, rows);  // (of ST2 too; RB - 1 in its place would read past the last wave's ring, and LDS)
  const int red_at = (SIZED ? rows : RB) * RP, red_bytes = align128(2 * W * red_at * 4);  // a wave's partial sums of an item, all of two items
  const int acc_bytes = max(red_bytes, align128(W * (SIZED ? p.T : TMAX) * R2 * 4));
  const int ringw1 = (LDS - lists - red_bytes) / W / 128 * 128, ringw2 = (LDS - lists - acc_bytes) / W / 128 * 128;
  const int S1 = min(MOST1, ringw1 / bytes1), S2 = min(MOST2, ringw2 / bytes2);
  const int tiles1 = p.f / PR1, n1 = nblk * tiles1, n2 = (p.d + R2 - 1) / R2;
  auto count = [&](int first, int n) { return first < n ? (n - 1 - first) / G + 1 : 0; };  // items first, first + G, ..
  auto block = [&](int b) {  // (uniform)
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(&s_blk[b]);
    return __builtin_bit_cast(Block, u32x2_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)v[0]),
                                             (uint32_t)__builtin_amdgcn_readfirstlane((int)v[1])});
  };
  // Phase-1 items: block bi's share of the tiles; a channel tile's blocks follow one
  // another, then the next tile's.  Moved on by G items with adds alone.
  const int g_blk = G / tiles1, g_tile = G - g_blk * tiles1;
  struct Item {
    int i, bi, at;  // bi * tiles1 + at = i
  };
  auto first_item = [&](int i) { return Item{i, i / tiles1, i % tiles1}; };
  auto next_item = [&](Item& m) {
    m.i += G, m.bi += g_blk, m.at += g_tile;
    if (m.at >= tiles1) m.at -= tiles1, ++m.bi;
  };
  auto item1 = [&](const Item& m, Block& b, int& tile) {
    b = block(m.bi);
    tile = m.at;
    if (TMAX > RB && b.nb > 1) {
      const int local = b.off * tiles1 + m.at;
      tile = local / b.nb;
      b = block(m.bi - b.off + local % b.nb);
    }
  };

  float* red = reinterpret_cast<float*>(pool);
  float* yacc = reinterpret_cast<float*>(pool);
  bool lost = false;  // the other workgroups' h did not come: see below
  int nmore = 0;

  // Sums of an item of phase 2 over the waves, and their stores.
  auto store_y = [&](int tile) {
    const int chans = min(R2, p.d - tile * R2);
    for (int i = tid; i < p.T * (R2 / 2); i += NT) {
      const int t = i / (R2 / 2), c = (i % (R2 / 2)) * 2;
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        a += yacc[(w * p.T + t) * R2 + c];
        b += yacc[(w * p.T + t) * R2 + c + 1];
      }
      if (c < chans)
        *reinterpret_cast<uint32_t*>(p.y + (int64_t)t * p.d + tile * R2 + c) = lost ? 0x7fc07fc0u : pack_bf2(a, b);
    }
  };

  if (wave == W) {  // ---- the serving wave
    bool take = true;
    for (int cur = vid;;) {
      Item m = first_item(cur);
#pragma nounroll
      for (int n = 0; m.i < n1; next_item(m), ++n) {
        Block b;
        int tile;
        item1(m, b, tile);
        lds_barrier();  // the item's partial sums are in red[n % 2]
        const float* rd = red + (n & 1) * W * red_at;
        // Lane l: row l / 16 of four, row l % 16 (8 gate, 8 up) of a 16-row tile.
        for (int i = 0; i < b.n * (R1 / 16); i += 4) {
          const int j = i + q, row = j / (R1 / 16), t = j % (R1 / 16);
          float v = 0.f;
          if (row < b.n) {
#pragma unroll
            for (int w = 0; w < W; ++w) v += rd[w * red_at + row * RP + 16 * t + r];
          }
          const float up = __shfl_xor(v, 8, WAVE), hv = v * sigmoidf_(v) * up, other = __shfl_xor(hv, 1, WAVE);
          if (row < b.n && r < 8 && r % 2 == 0)
            __hip_atomic_store(reinterpret_cast<uint32_t*>(p.h + (int64_t)(s_row[b.pos + row] & 0xffff) * p.f + tile * PR1 +
                                                           8 * t + r),
                               pack_bf2(hv, other), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
      // h was stored past the XCD's L2 (atomic, at agent scope), so its stores being
      // complete is enough: a release fence writes back the whole L2, which took
      // 1 to 6 us with the CUs of an XCD at it together.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (lane == 0)
        __hip_atomic_store(p.sync + SYNC_FLAGS + cur, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // All flags up: on.  Else, after 20 us, take the number of a workgroup that
      // has not started, if there is one.  (So many looks, 1 to 2 us each, pass only
      // where the workspace's rule is broken, and another call has cleared the flags: y
      // is then NaN, and the kernel ends.  Looks and not time: the clock runs on while
      // a queue is off the GPU.)
      int cmd = -1;
      const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
      for (int looks = 0;; ++looks) {
        bool all = true;
        for (int i = lane; i < G; i += 64)
          all &= __hip_atomic_load(p.sync + SYNC_FLAGS + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0;
        if (__all(all)) break;
        const uint64_t dt = __builtin_amdgcn_s_memrealtime() - t0;  // 10 ns each
        if (take && dt > 2000 && nmore < 256) {
          int v = 0;
          if (lane == 0) v = (int)__hip_atomic_fetch_add(p.sync, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          v = __builtin_amdgcn_readfirstlane(v);
          if (v < G) {
            cmd = v;
            break;
          }
          take = false;
        }
        if (looks >= 1 << 23) {
          cmd = -2;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      if (lane == 0) {
        s_cmd = cmd;
        if (cmd >= 0) s_more[nmore] = (uint16_t)cmd;
      }
      lds_barrier();  // (1)
      lost = cmd == -2;
      if (cmd < 0) break;
      ++nmore;
      cur = cmd;
      lds_barrier();  // (2): s_cmd is read
    }
    for (int l = 0; l <= nmore; ++l)
      for (int item = l ? s_more[l - 1] : vid; item < n2; item += G) {
        lds_barrier();
        store_y(item);
        lds_barrier();
      }
    return;
  }

  // ---- a streaming wave
  // (What only the start of an item needs is read from the arguments there, not
  // kept in scalar registers, of which the loops have too few: spilled ones cost
  // a vector instruction each time.)
  typedef const __attribute__((address_space(4))) DecodeParams* Args;
  auto args = [&]() {
    Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return a;
  };
  // (Phase 2's rings may lie over other waves' of phase 1: a wave copies into its own
  // after the last barrier of phase 1, when all have read theirs.)
  const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)pool);
  const uint32_t ring1 = base + red_bytes + wave * ringw1, ring2 = base + acc_bytes + wave * ringw2;
  const uint8_t *ring1_p = pool + red_bytes + wave * ringw1, *ring2_p = pool + acc_bytes + wave * ringw2;
  Ages ages;

  // Phase 2's share: of the item's stages (blocks by stages of a row of f) a
  // stretch, the same in every item.
  const int C2 = (p.f + ST2::KS - 1) / ST2::KS, q0 = nblk * C2 * wave / W, per2 = nblk * C2 * (wave + 1) / W - q0;
  const int blk2 = q0 / C2, st2 = q0 - blk2 * C2;  // where it starts
  Source src;
  uint32_t xr2[ST2::XI];
  int rows2 = 0;
  auto source2 = [&](int item, int blk) {
    const Args a = args();
    const int d = a->d, f = a->f;
    const int64_t pitch = GRP ? f / 2 : (int64_t)f * 2;
    const Block b = block(blk);
    const int64_t row = (int64_t)b.e * d + item * R2;
    src.rows = min(R2, d - item * R2);
    src.w[0] = make_rsrc(a->w2 + row * pitch, src.rows * pitch);
    src.pitch = (uint32_t)pitch;
    if (GRP) {
      const int groups = (f + GRP - 1) / (GRP ? GRP : 1);
      src.s[0] = make_rsrc(a->s2 + row * groups, (uint64_t)src.rows * groups * 4);
      src.spitch = groups * 4;
    }
    src.x = make_rsrc(a->h, (uint64_t)(a->T * a->k) * f * 2);
    src.K = f;
    rows2 = b.n;
#pragma unroll
    for (int n = 0; n < ST2::XI; ++n)
      xr2[n] = (s_row[b.pos + min(ST2::x_row(n, lane), b.n - 1)] & 0xffff) * (uint32_t)f * 2;
  };
  // The stage to copy next in phase 2.
  int c_item = vid, c_blk = blk2, c_st = st2, c_left = per2;
  bool c_new = true;
  auto next2 = [&]() {
    c_new = false;
    if (--c_left == 0) c_left = per2, c_item += G, c_blk = blk2, c_st = st2, c_new = true;
    else if (++c_st == C2) c_st = 0, ++c_blk, c_new = true;
  };

  int ahead = 0;  // stages of phase 2 whose weights were asked for before all of h was there
  for (int cur = vid;;) {
    // Phase 1: the wave has a stretch of d in every item.
    const int C1 = (p.d + ST1::KS - 1) / ST1::KS, s0 = C1 * wave / W, per1 = C1 * (wave + 1) / W - s0;
    const int items = count(cur, n1);
    if (per1 == 0) {
#pragma nounroll
      for (int n = 0; n < items; ++n) {
        float* rd = red + ((n & 1) * W + wave) * red_at;
        for (int i = lane; i < red_at; i += 64) rd[i] = 0.f;
        lds_barrier();
      }
    } else {
      uint32_t xr1[ST1::XI];
      int rows1 = 0, c_at = 0;  // copied next: stage of the item, item
      Item c_m = first_item(cur);
      int u_at = 0, u_n = 0, head = 0, tail = 0;  // used next: stage of the item, item's place; ring slots
      f32x4_t acc[ST1::RT];
#pragma unroll
      for (int t = 0; t < ST1::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      src.pitch = (uint32_t)(GRP ? p.d / 2 : p.d * 2);
      src.K = p.d, src.rows = PR1;
      src.x = make_rsrc(p.x, (uint64_t)p.T * p.d * 2);
      auto copy = [&]() {
                  if (c_at == 0) {
                    const Args a = args();
                    const int d = a->d;
                    Block b;
                    int tile;
                    item1(c_m, b, tile);
                    const int64_t row = (int64_t)b.e * a->f + tile * PR1, pitch = GRP ? d / 2 : (int64_t)d * 2;
                    src.w[0] = make_rsrc(a->w1 + row * pitch, PR1 * pitch);
                    src.w[1] = make_rsrc(a->w3 + row * pitch, PR1 * pitch);
                    if (GRP) {
                      const int groups = (d + GRP - 1) / (GRP ? GRP : 1);
                      src.s[0] = make_rsrc(a->s1 + row * groups, (uint64_t)PR1 * groups * 4);
                      src.s[1] = make_rsrc(a->s3 + row * groups, (uint64_t)PR1 * groups * 4);
                      src.spitch = groups * 4;
                    }
                    rows1 = b.n;
        #pragma unroll
                    for (int n = 0; n < ST1::XI; ++n)
                      xr1[n] = (s_row[b.pos + min(ST1::x_row(n, lane), b.n - 1)] >> 16) * (uint32_t)d * 2;
                  }
                  const int k0 = (s0 + c_at) * ST1::KS;
                  const uint32_t at = __builtin_amdgcn_readfirstlane(ring1 + head * bytes1);
                  ST1::copy_w(src, k0, at, lane);
                  ages.push(PRE1 + ST1::copy_x(src, xr1, rows1, k0, at, lane));
                  head = head + 1 == S1 ? 0 : head + 1;
                  if (++c_at == per1) c_at = 0, next_item(c_m);
      };
#pragma nounroll
      while (ages.n < S1 && c_m.i < n1) copy();
#pragma nounroll
      while (u_n < items) {
        ages.pop();
        wait_younger<(MOST1 - 1) * (PRE1 + 1)>(ages.sum);
        ST1 s;
        s.read(ring1_p + tail * bytes1, lane, col);
        if (!ST1::EARLY) s.multiply(acc, lane);
        reads_done();
        tail = tail + 1 == S1 ? 0 : tail + 1;
        if (c_m.i < n1) copy();
        if (ST1::EARLY) s.multiply(acc, lane);
        if (++u_at == per1) {
          float* rd = red + ((u_n & 1) * W + wave) * red_at;
          if (r < (SIZED ? rows : RB)) {
#pragma unroll
            for (int t = 0; t < ST1::RT; ++t) *reinterpret_cast<f32x4_t*>(rd + r * RP + 16 * t + 4 * q) = acc[t];
          }
#pragma unroll
          for (int t = 0; t < ST1::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          u_at = 0;
          ++u_n;
          lds_barrier();
        }
      }
    }
    // The weights of phase 2's first stages, while the other workgroups finish theirs.
    if (cur == vid) {
      ahead = min(S2, count(vid, n2) * per2);
#pragma nounroll
      for (int i = 0; i < ahead; ++i) {
        if (c_new) source2(c_item, c_blk);
        ST2::copy_w(src, c_st * ST2::KS, __builtin_amdgcn_readfirstlane(ring2 + i * bytes2), lane);
        next2();
      }
    }
    lds_barrier();  // (1)
    const int cmd = __builtin_amdgcn_readfirstlane(s_cmd);
    lost = cmd == -2;
    if (cmd < 0) break;
    ++nmore;  // a number taken over; what was copied ahead is dropped
    cur = cmd;
    // (before the barrier: it may lie over other waves' rings of phase 1)
    wait_vm<0>();
    asm volatile("" ::: "memory");
    lds_barrier();  // (2)
    ahead = 0;
  }

  // Phase 2.
#pragma nounroll
  for (int l = 0; l <= nmore; ++l) {
    const int first = __builtin_amdgcn_readfirstlane(l ? (int)s_more[l - 1] : vid);
    c_item = first, c_blk = blk2, c_st = st2, c_left = per2, c_new = true;
    int head = 0, tail = 0;
#pragma nounroll
    for (; head < ahead; ++head) {  // their rows of h
      if (c_new) source2(c_item, c_blk);
      ages.push(ST2::copy_x(src, xr2, rows2, c_st * ST2::KS, __builtin_amdgcn_readfirstlane(ring2 + head * bytes2), lane));
      next2();
    }
    ahead = 0;
    if (head == S2) head = 0;
    const int items = count(first, n2);
    int copies = items * per2 - ages.n;  // stages that are still to be copied
    float* mine = yacc + wave * p.T * R2;
    auto copy = [&]() {
      if (c_new) source2(c_item, c_blk);
      const uint32_t at = __builtin_amdgcn_readfirstlane(ring2 + head * bytes2);
      const int k0 = c_st * ST2::KS;
      ST2::copy_w(src, k0, at, lane);
      ages.push(PRE2 + ST2::copy_x(src, xr2, rows2, k0, at, lane));
      next2();
      head = head + 1 == S2 ? 0 : head + 1;
      --copies;
    };
#pragma nounroll
    while (ages.n < S2 && copies > 0) copy();
#pragma nounroll
    for (int n = 0; n < items; ++n) {
      for (int i = lane; i < p.T * R2; i += 64) mine[i] = 0.f;
      f32x4_t acc[ST2::RT];
#pragma unroll
      for (int t = 0; t < ST2::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      int blk = blk2, st = st2;
#pragma nounroll
      for (int left = per2; left > 0;) {
        ages.pop();
        wait_younger<(MOST2 - 1) * (PRE2 + 1)>(ages.sum);
        ST2 s;
        s.read(ring2_p + tail * bytes2, lane, col);
        if (!ST2::EARLY) s.multiply(acc, lane);
        reads_done();
        tail = tail + 1 == S2 ? 0 : tail + 1;
        if (copies > 0) copy();
        if (ST2::EARLY) s.multiply(acc, lane);
        --left;
        if (++st == C2 || left == 0) {  // the block's products, times the routing weights, to their tokens
          const Block b = block(blk);
          if (r < b.n) {
            const int token = s_row[b.pos + r] >> 16;
            const float w = s_roww[b.pos + r];
            float* to = mine + token * R2 + 4 * q;
#pragma unroll
            for (int t = 0; t < ST2::RT; ++t)
              if (R2 - 16 * t >= 16 || q < 2) {
                f32x4_t v = *reinterpret_cast<f32x4_t*>(to + 16 * t);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += w * acc[t][i];
                *reinterpret_cast<f32x4_t*>(to + 16 * t) = v;
              }
          }
#pragma unroll
          for (int t = 0; t < ST2::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          st = 0;
          ++blk;
        }
      }
      lds_barrier();
      store_y(first + n * G);
      lds_barrier();
    }
  }
}

// ---------------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }
// Parts of d in the logits' partial sums (1 or 4, see route_token): more of them
// spread the router's weights over more CUs (64 tokens, 384 experts of 6144: 24 us
// with one part, 9 with four).
int router_parts(const moe_desc& d) { return d.d >= 1024 ? 4 : 1; }
int64_t part_bytes(const moe_desc& d) { return align256((int64_t)router_parts(d) * d.T * d.E * 4); }
constexpr int64_t SYNC_BYTES = 4096;
constexpr int MAX_WGS = 256;  // (a workgroup may take over all the others' numbers)

template <int GRP, int TMAX, int RB, int R1, int R2, int SUB2, int W>
hipError_t run(const DecodeParams& p, int grid, hipStream_t s) {
  decode_kernel<GRP, TMAX, RB, R1, R2, SUB2, W><<<(unsigned)grid, 64 * (W + 1), 0, s>>>(p);
  return hipGetLastError();
}

template <int GRP>
hipError_t decode(const DecodeParams& p, int grid, hipStream_t s) {
  // Channels of d an item: 24 where that leaves no workgroup with more than 8 would.
  auto busiest = [&](int r2) { return ((p.d + r2 - 1) / r2 + grid - 1) / grid * r2; };
  const bool wide = busiest(24) <= busiest(8);
  if constexpr (GRP == 0) {
    if (p.T <= 2) return wide ? run<0, 2, 2, 16, 24, 1, 8>(p, grid, s) : run<0, 2, 2, 16, 8, 3, 8>(p, grid, s);
    if (p.T <= 16) return wide ? run<0, 16, 16, 16, 24, 1, 8>(p, grid, s) : run<0, 16, 16, 16, 8, 2, 8>(p, grid, s);
    return wide ? run<0, MAX_T, 12, 16, 24, 1, 8>(p, grid, s) : run<0, MAX_T, 12, 16, 8, 2, 8>(p, grid, s);
  } else {
    // (twelve waves where their registers hold a stage of the smaller groups' scales too)
    constexpr int W2 = GRP == 128 ? 12 : 8;
    if (p.T <= 2) return wide ? run<GRP, 2, 2, 32, 24, 1, W2>(p, grid, s) : run<GRP, 2, 2, 32, 8, 1, W2>(p, grid, s);
    // 16 channels of f an item where that leaves four items and more to a workgroup.
    if (p.T <= 16 && (int64_t)std::min(p.NL, p.T * p.k) * (p.f / 16) >= 4 * grid)
      return wide ? run<GRP, 16, 4, 32, 24, 1, 8>(p, grid, s) : run<GRP, 16, 4, 32, 8, 1, 8>(p, grid, s);
    if (p.T <= 16) return wide ? run<GRP, 16, 4, 16, 24, 1, 8>(p, grid, s) : run<GRP, 16, 4, 16, 8, 1, 8>(p, grid, s);
    // Eight rows a block.  In turn on one card, 64 tokens of 64 experts (2048 x 1024), of 96
    // (6144 x 1792) and of 384, 96 of them here: 139, 461 and 281 us, and 24 tokens 94, 331
    // and 171; with four rows 196, 617 and 276, 101, 341 and 167; with twelve, whose sums
    // leave the rings less room, 116, 431 and 284, 96, 336 and 173.
    return wide ? run<GRP, MAX_T, 8, 32, 24, 1, 8>(p, grid, s) : run<GRP, MAX_T, 8, 32, 8, 1, 8>(p, grid, s);
  }
}

}  // namespace

size_t decode_workspace(const moe_desc& d) {
  return (size_t)(SYNC_BYTES + part_bytes(d) + (int64_t)d.T * d.k * d.f * 2);
}

hipError_t launch_decode(const moe_desc& d, int group, int n_groups, const void* x, const void* Wr, const float* bias,
                         const void* W1, const float* W1s, const void* W3, const float* W3s, const void* W2,
                         const float* W2s, int32_t* idx, float* w, void* y, void* ws, hipStream_t s) {
  uint32_t* sync = reinterpret_cast<uint32_t*>(ws);
  float* part = reinterpret_cast<float*>((char*)ws + SYNC_BYTES);
  uint16_t* h = reinterpret_cast<uint16_t*>((char*)ws + SYNC_BYTES + part_bytes(d));
  const int grid = std::min(num_cus(), MAX_WGS);
  const int ks = router_parts(d);
  const dim3 rgrid = Wr ? dim3((unsigned)((d.E + 15) / 16), (unsigned)ks) : dim3(1, 1);
  if (d.T <= 16)
    decode_router_kernel<1><<<rgrid, 1024, 0, s>>>((const uint16_t*)x, (const uint16_t*)Wr, d.T, d.d, d.E, part, sync,
                                                  SYNC_FLAGS + grid);
  else
    decode_router_kernel<4><<<rgrid, 1024, 0, s>>>((const uint16_t*)x, (const uint16_t*)Wr, d.T, d.d, d.E, part, sync,
                                                  SYNC_FLAGS + grid);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const DecodeParams p{(const uint16_t*)x, (const uint8_t*)W1, (const uint8_t*)W3, (const uint8_t*)W2, W1s, W3s, W2s,
                       Wr ? part : nullptr, bias, idx, w, h, (uint16_t*)y, sync, d.T, d.d, d.f, d.E, d.k, d.expert_begin,
                       d.num_local, d.renormalize, n_groups, ks};
  switch (group) {
    case 0: return decode<0>(p, grid, s);
    case 32: return decode<32>(p, grid, s);
    case 64: return decode<64>(p, grid, s);
    default: return decode<128>(p, grid, s);
  }
}

}  // namespace moe
