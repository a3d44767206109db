// The whole expert layer for a few tokens (T <= 64) in two kernels: the router
// logits, then everything else.
//
// At these sizes the layer streams the weights of the experts that the tokens
// take, each byte once, and is bound by HBM; the rest is latency.  The second
// kernel therefore has one workgroup per CU, whose waves copy weights from
// start to end (stream.h): every workgroup selects for all tokens by itself
// (a few hundred logits each, cheaper than a kernel or a hand-over), then
//   phase 1: (expert, 8 channels of f or more) items: gate and up rows over all
//            of d, h = silu(G) U to memory as bf16,
//   phase 2: (8 or 16 channels of d) items: for every expert hit, its W2 rows
//            over all of f, times the routing weights, summed over the experts
//            in LDS, so that y is written once and no atomics change its order.
// Between the phases all of h has to be there.  Each workgroup raises a flag
// when its phase-1 items are done and waits for all flags; the W2 copies of its
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
constexpr int SYNC_FLAGS = 64;  // sync[0]: the counter of workgroups; sync[SYNC_FLAGS + i]: number i's phase 1 is done

// ---------------------------------------------------------------------------
// Router logits
// ---------------------------------------------------------------------------

// Partial sums part[ks][t][e] of x Wr^T: a workgroup has 16 experts and a
// gridDim.y-th of d, a wave a quarter of that; 16 CT tokens.  Clears the second
// kernel's counter and flags.
template <int CT>
__global__ void __launch_bounds__(256) decode_router_kernel(const uint16_t* __restrict__ x,
                                                            const uint16_t* __restrict__ wr, int T, int d, int E,
                                                            float* __restrict__ part, uint32_t* __restrict__ sync,
                                                            int nsync) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  __shared__ float red[4][CT * 16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < nsync; i += 256) sync[i] = 0;
  if (!wr) return;  // (the routing is given)
  const int steps = d / 32, parts = gridDim.y * 4, me = blockIdx.y * 4 + wave;
  const int s0 = steps * me / parts, s1 = steps * (me + 1) / parts;
  const uint16_t* a = wr + (int64_t)min((int)blockIdx.x * 16 + r, E - 1) * d + q * 8;
  const uint16_t* b[CT];
  f32x4_t acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    b[c] = x + (int64_t)min(c * 16 + r, T - 1) * d + q * 8;
    acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  constexpr int U = CT == 1 ? 6 : 2;  // steps whose loads are in flight together
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
  for (int i = tid; i < CT * 256; i += 256) {
    const int t = i >> 4, e = (int)blockIdx.x * 16 + (i & 15);
    if (t < T && e < E)
      part[((int64_t)blockIdx.y * T + t) * E + e] =
          (red[0][t][i & 15] + red[1][t][i & 15]) + (red[2][t][i & 15] + red[3][t][i & 15]);
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

// The tokens that one pass over an expert's rows serves.
struct alignas(8) Block {
  uint16_t e, n;   // local expert; tokens (<= RB)
  uint16_t pos;    // their place in the list of rows
  uint8_t off, nb; // which of the expert's blocks it is, and of how many
};

template <int MAXV>
__device__ __forceinline__ void route_token(const DecodeParams& p, int t, int lane, int32_t* idx, float* w, int32_t* si,
                                            float* sv) {
  float v[MAXV];
#pragma unroll
  for (int i = 0; i < MAXV; ++i) v[i] = i * 64 + lane < p.E ? (p.bias ? p.bias[i * 64 + lane] : 0.f) : -INFINITY;
  for (int s = 0; s < p.ks; ++s) {
    const float* row = p.part + ((int64_t)s * p.T + t) * p.E;
#pragma unroll
    for (int i = 0; i < MAXV; ++i)
      if (i * 64 + lane < p.E) v[i] += row[i * 64 + lane];
  }
  if (p.n_groups > 1) topk_rounds<MAXV, true>(v, lane, t, p.E, p.k, p.renorm, p.n_groups, idx, w);
  else topk_token<MAXV>(v, lane, t, p.E, p.k, p.renorm, idx, w, si, sv);
}

// GRP 0: bf16 weights.  TMAX tokens at most, RB of them in a pass.  R1 rows (half
// gate, half up) by 128 bytes a stage in phase 1, R2 by SUB2 times 128 in phase 2.
template <int GRP, int TMAX, int RB, int R1, int R2, int SUB2, int W, int S>
__global__ void __launch_bounds__(64 * (W + 1)) decode_kernel(DecodeParams p) {
  using namespace stream;
  using ST1 = Stage<GRP, R1, 1, true, RB>;
  using ST2 = Stage<GRP, R2, SUB2, false, RB>;
  constexpr int SLOT = ST1::BYTES > ST2::BYTES ? ST1::BYTES : ST2::BYTES;
  constexpr int PER1 = ST1::WI + ST1::SI + ST1::XI, PRE2 = ST2::WI + ST2::SI, PER2 = PRE2 + ST2::XI;
  constexpr int RP = R1 + 4;  // pitch of phase 1's partial sums (floats)
  constexpr int RED = 2 * W * RB * RP * 4, YACC = W * TMAX * R2 * 4, ACC = RED > YACC ? RED : YACC;
  constexpr int RING = W * S * SLOT;
  constexpr int ROWS = TMAX * MAX_K, BLOCKS = TMAX <= RB ? (ROWS < MAX_E ? ROWS : MAX_E) : MAX_E + ROWS / RB;
  // Scratch of the selection, over the ring before it starts.
  constexpr int O_IDX = 0, O_W = O_IDX + ROWS * 4, O_MASK = O_W + ROWS * 4, O_BASE = O_MASK + MAX_E * 8,
                O_TOP = O_BASE + MAX_E * 2, SCRATCH = O_TOP + (W + 1) * 512;
  static_assert(SCRATCH <= RING, "scratch");
  static_assert((S - 1) * PER1 < 64 && (S - 1) * PER2 < 64, "vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t ring_m[RING];
  __shared__ __attribute__((aligned(16))) uint8_t acc_m[ACC];
  __shared__ Block s_blk[BLOCKS];
  __shared__ float s_roww[ROWS];
  __shared__ uint16_t s_row[ROWS];  // slots of the rows, by expert
  __shared__ uint16_t s_more[256];  // numbers taken over
  __shared__ int s_vid, s_nblk, s_cmd;

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = gridDim.x, slots = p.T * p.k;

  // ---- the selection, and the rows by expert
  int32_t* l_idx = reinterpret_cast<int32_t*>(ring_m + O_IDX);
  float* l_w = reinterpret_cast<float*>(ring_m + O_W);
  unsigned long long* l_mask = reinterpret_cast<unsigned long long*>(ring_m + O_MASK);
  uint16_t* l_base = reinterpret_cast<uint16_t*>(ring_m + O_BASE);
  if (tid == 64 * W)
    s_vid = (int)__hip_atomic_fetch_add(p.sync, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < slots; i += 64 * (W + 1)) {
    // (a token whose logits are not numbers may leave slots unwritten)
    l_idx[i] = p.part ? i % p.k : p.idx[i];
    l_w[i] = p.part ? __uint_as_float(0x7fc00000u) : p.w[i];
  }
  for (int i = tid; i < p.NL; i += 64 * (W + 1)) l_mask[i] = 0;
  __syncthreads();
  if (p.part) {
    int32_t* si = reinterpret_cast<int32_t*>(ring_m + O_TOP + wave * 512);
    float* sv = reinterpret_cast<float*>(si + 64);
    for (int t = wave; t < p.T; t += W + 1) {
      if (p.E <= 64) route_token<1>(p, t, lane, l_idx, l_w, si, sv);
      else if (p.E <= 128) route_token<2>(p, t, lane, l_idx, l_w, si, sv);
      else if (p.E <= 384) route_token<6>(p, t, lane, l_idx, l_w, si, sv);
      else route_token<16>(p, t, lane, l_idx, l_w, si, sv);
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i < slots; i += 64 * (W + 1)) p.idx[i] = l_idx[i], p.w[i] = l_w[i];
  }
  const int vid = __builtin_amdgcn_readfirstlane(s_vid);
  if (vid >= G) return;  // (another workgroup has done this one's items)
  for (int i = tid; i < slots; i += 64 * (W + 1)) {
    const uint32_t e = (uint32_t)l_idx[i] - (uint32_t)p.e0;
    if (e < (uint32_t)p.NL) atomicOr(&l_mask[e], 1ull << (i / p.k));
  }
  __syncthreads();
  if (wave == 0) {  // exclusive sums of the experts' rows and blocks, 64 experts at a time
    uint32_t before = 0;
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
      for (int b = 0; b < nb; ++b)
        s_blk[(ex >> 16) + b] = Block{(uint16_t)e, (uint16_t)min(RB, n - b * RB), (uint16_t)((ex & 0xffff) + b * RB),
                                      (uint8_t)b, (uint8_t)nb};
      before += __shfl(inc, 63, WAVE);
    }
    if (lane == 0) s_nblk = (int)(before >> 16);
  }
  __syncthreads();
  for (int i = tid; i < slots; i += 64 * (W + 1)) {
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
    s_row[pos] = (uint16_t)i;
    s_roww[pos] = w;
  }
  __syncthreads();

  // ---- items
  constexpr int PR1 = R1 / 2;
  const int nblk = __builtin_amdgcn_readfirstlane(s_nblk);
  const int tiles1 = p.f / PR1, n1 = nblk * tiles1, n2 = p.d / R2;
  const int C1 = (p.d + ST1::KS - 1) / ST1::KS, C2 = (p.f + ST2::KS - 1) / ST2::KS;  // stages of a row
  const int64_t pitch1 = GRP ? p.d / 2 : (int64_t)p.d * 2, pitch2 = GRP ? p.f / 2 : (int64_t)p.f * 2;
  const int groups1 = GRP ? (p.d + GRP - 1) / (GRP ? GRP : 1) : 0, groups2 = GRP ? (p.f + GRP - 1) / (GRP ? GRP : 1) : 0;
  auto block = [&](int b) {  // (uniform)
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(&s_blk[b]);
    return __builtin_bit_cast(Block, u32x2_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)v[0]),
                                             (uint32_t)__builtin_amdgcn_readfirstlane((int)v[1])});
  };
  // Phase-1 item i: a channel tile's blocks follow one another, then the next tile's.
  auto item1 = [&](int i, Block& b, int& tile) {
    const int bi = i / tiles1;
    b = block(bi);
    const int b0 = bi - b.off, local = i - b0 * tiles1;
    tile = local / b.nb;
    b = block(b0 + local % b.nb);
  };

  float* red = reinterpret_cast<float*>(acc_m);
  float* yacc = reinterpret_cast<float*>(acc_m);
  bool lost = false;  // the other workgroups' h did not come: see below
  int nmore = 0;

  // Sums of an item of phase 2 over the waves, and their stores.
  auto store_y = [&](int tile) {
    for (int i = tid; i < p.T * (R2 / 2); i += 64 * (W + 1)) {
      const int t = i / (R2 / 2), c = (i % (R2 / 2)) * 2;
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        a += yacc[(w * p.T + t) * R2 + c];
        b += yacc[(w * p.T + t) * R2 + c + 1];
      }
      *reinterpret_cast<uint32_t*>(p.y + (int64_t)t * p.d + tile * R2 + c) = lost ? 0x7fc07fc0u : pack_bf2(a, b);
    }
  };

  if (wave == W) {  // ---- the serving wave
    bool take = true;
    for (int cur = vid;;) {
      for (int item = cur, n = 0; item < n1; item += G, ++n) {
        Block b;
        int tile;
        item1(item, b, tile);
        lds_barrier();  // the item's partial sums are in red[n % 2]
        const float* rd = red + (n & 1) * W * RB * RP;
        for (int i = lane; i < b.n * (PR1 / 2); i += 64) {
          const int row = i / (PR1 / 2), c = (i % (PR1 / 2)) * 2, at = row * RP + (c / 8) * 16 + c % 8;
          float g[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              g[j] += rd[w * RB * RP + at + j];
              u[j] += rd[w * RB * RP + at + 8 + j];
            }
          const uint32_t hv = pack_bf2(g[0] * sigmoidf_(g[0]) * u[0], g[1] * sigmoidf_(g[1]) * u[1]);
          __hip_atomic_store(reinterpret_cast<uint32_t*>(p.h + (int64_t)s_row[b.pos + row] * p.f + tile * PR1 + c), hv,
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
      if (lane == 0)
        __hip_atomic_store(p.sync + SYNC_FLAGS + cur, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // All flags up: on.  Else, after 20 us, take the number of a workgroup that
      // has not started, if there is one.  (Ten seconds pass only where the
      // workspace's rule is broken, and another call has cleared the flags: y is
      // then NaN, and the kernel ends.)
      int cmd = -1;
      const uint64_t t0 = __builtin_amdgcn_s_memrealtime();
      for (;;) {
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
        if (dt > 1000000000ull) {
          cmd = -2;
          break;
        }
        __builtin_amdgcn_s_sleep(2);
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
  const uint32_t ring = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring_m) + wave * S * SLOT;
  const uint8_t* ring_p = ring_m + wave * S * SLOT;
  // What is copied next: phase (3: nothing), item, block, stage.
  int c_ph = 1, c_item = vid, c_blk = 0, c_st = wave, c_step = G;
  bool c_new = true, c_on = true, h_there = false;  // c_on: phase 2 follows
  Source src;
  uint32_t xr1[ST1::XI], xr2[ST2::XI];
  int head = 0, tail = 0, flying = 0;  // ring slots; stages in flight

  auto source1 = [&]() {
    Block b;
    int tile;
    item1(c_item, b, tile);
    const int64_t row = (int64_t)b.e * p.f + tile * PR1;
    src.w[0] = make_rsrc(p.w1 + row * pitch1, PR1 * pitch1);
    src.w[1] = make_rsrc(p.w3 + row * pitch1, PR1 * pitch1);
    if (GRP) {
      src.s[0] = make_rsrc(p.s1 + row * groups1, (uint64_t)PR1 * groups1 * 4);
      src.s[1] = make_rsrc(p.s3 + row * groups1, (uint64_t)PR1 * groups1 * 4);
    }
    src.x = make_rsrc(p.x, (uint64_t)p.T * p.d * 2);
    src.pitch = (uint32_t)pitch1, src.spitch = groups1 * 4, src.K = p.d, src.rows = PR1;
#pragma unroll
    for (int n = 0; n < ST1::XI; ++n) {
      const int row = ST1::x_row(n, lane);
      xr1[n] = row < b.n ? (uint32_t)(s_row[b.pos + row] / p.k) * (uint32_t)p.d * 2 : NOWHERE;
    }
  };
  auto source2 = [&](int item, int blk) {
    const Block b = block(blk);
    const int64_t row = (int64_t)b.e * p.d + item * R2;
    src.w[0] = make_rsrc(p.w2 + row * pitch2, R2 * pitch2);
    if (GRP) src.s[0] = make_rsrc(p.s2 + row * groups2, (uint64_t)R2 * groups2 * 4);
    src.x = make_rsrc(p.h, (uint64_t)slots * p.f * 2);
    src.pitch = (uint32_t)pitch2, src.spitch = groups2 * 4, src.K = p.f, src.rows = R2;
#pragma unroll
    for (int n = 0; n < ST2::XI; ++n) {
      const int row = ST2::x_row(n, lane);
      xr2[n] = row < b.n ? (uint32_t)s_row[b.pos + row] * (uint32_t)p.f * 2 : NOWHERE;
    }
  };
  // To the next stage of phase 2 that this wave has; false past the last item.
  auto settle2 = [&](int& item, int& blk, int& st, bool& fresh) {
    if (nblk == 0) return false;
    while (item < n2 && st >= C2) {
      st -= C2;
      fresh = true;
      if (++blk == nblk) blk = 0, st = wave, item += c_step;
    }
    return item < n2;
  };
  auto copy_next = [&]() {
    if (c_ph == 1) {
      while (c_item < n1 && c_st >= C1) c_item += G, c_st = wave, c_new = true;
      if (c_item >= n1) c_ph = c_on ? 2 : 3, c_item = vid, c_blk = 0, c_st = wave, c_new = true;
    }
    if (c_ph == 2 && !settle2(c_item, c_blk, c_st, c_new)) c_ph = 3;
    if (c_ph == 3) return;
    const uint32_t at = __builtin_amdgcn_readfirstlane(ring + head * SLOT);
    if (c_ph == 1) {
      if (c_new) source1();
      const int k0 = __builtin_amdgcn_readfirstlane(c_st * ST1::KS);
      ST1::copy_w(src, k0, at, lane);
      ST1::copy_x(src, xr1, k0, at, lane);
    } else {
      if (c_new) source2(c_item, c_blk);
      const int k0 = __builtin_amdgcn_readfirstlane(c_st * ST2::KS);
      ST2::copy_w(src, k0, at, lane);
      if (h_there) ST2::copy_x(src, xr2, k0, at, lane);
    }
    c_new = false;
    c_st += W;
    head = head + 1 == S ? 0 : head + 1;
    ++flying;
  };
  auto taken = [&]() {
    tail = tail + 1 == S ? 0 : tail + 1;
    --flying;
  };

  for (int i = 0; i < S; ++i) copy_next();
  for (int cur = vid;;) {
    for (int item = cur, n = 0; item < n1; item += G, ++n) {
      f32x4_t acc[ST1::RT];
#pragma unroll
      for (int t = 0; t < ST1::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int st = wave; st < C1; st += W) {
        // the oldest stage has landed when no more than the S - 1 younger ones' copies are outstanding
        if (flying < S) wait_vm<0>();
        else if (c_ph == 1) wait_vm<(S - 1) * PER1>();
        else wait_vm<(S - 1) * (PRE2 < PER1 ? PRE2 : PER1)>();
        asm volatile("" ::: "memory");
        ST1 s;
        s.read(ring_p + tail * SLOT, lane);
        reads_done();
        taken();
        copy_next();
        s.multiply(acc);
      }
      float* rd = red + ((n & 1) * W + wave) * RB * RP;
      if (r < RB) {
#pragma unroll
        for (int t = 0; t < ST1::RT; ++t) *reinterpret_cast<f32x4_t*>(rd + r * RP + 16 * t + 4 * q) = acc[t];
      }
      lds_barrier();
    }
    lds_barrier();  // (1)
    const int cmd = __builtin_amdgcn_readfirstlane(s_cmd);
    lost = cmd == -2;
    if (cmd < 0) break;
    // A number taken over: what was copied ahead for phase 2 is dropped.
    ++nmore;
    cur = cmd;
    lds_barrier();  // (2)
    wait_vm<0>();
    asm volatile("" ::: "memory");
    head = tail = flying = 0;
    c_ph = 1, c_item = cur, c_blk = 0, c_st = wave, c_new = true, c_on = false;
    for (int i = 0; i < S; ++i) copy_next();
  }

  // Phase 2.  The stages in flight, if any, are its first ones without their rows of h.
  h_there = true;
  int late = 0;  // stages whose rows of h were copied after the weights of all in flight
  if (c_on) {
    const int ahead = flying;
    int item = vid, blk = 0, st = wave;
    for (int i = 0; i < ahead; ++i) {
      bool fresh = true;
      settle2(item, blk, st, fresh);
      source2(item, blk);
      ST2::copy_x(src, xr2, __builtin_amdgcn_readfirstlane(st * ST2::KS),
                  __builtin_amdgcn_readfirstlane(ring + ((tail + i) % S) * SLOT), lane);
      st += W;
    }
    late = ahead;
    c_new = true;
  }
  for (int l = 0; l <= nmore; ++l) {
    const int first = __builtin_amdgcn_readfirstlane(l ? (int)s_more[l - 1] : vid);
    if (l > 0 || !c_on) {
      c_ph = 2, c_item = first, c_blk = 0, c_st = wave, c_new = true;
      head = tail = flying = 0;
      for (int i = 0; i < S; ++i) copy_next();
    }
    for (int item = first; item < n2; item += G) {
      float* mine = yacc + wave * p.T * R2;
      for (int i = lane; i < p.T * R2; i += 64) mine[i] = 0.f;
      f32x4_t acc[1] = {{0.f, 0.f, 0.f, 0.f}};
      int have = -1;
      auto flush = [&]() {  // the block's products, times the routing weights, to their tokens
        if (have < 0) return;
        const Block b = block(have);
        if (r < b.n && (R2 > 8 || q < 2)) {
          const int slot = s_row[b.pos + r];
          const float w = s_roww[b.pos + r];
          f32x4_t* to = reinterpret_cast<f32x4_t*>(mine + (slot / p.k) * R2 + 4 * q);
          f32x4_t v = *to;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += w * acc[0][i];
          *to = v;
        }
        acc[0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      };
      for (int blk = 0, st = wave; blk < nblk;) {
        if (st >= C2) {
          st -= C2;
          ++blk;
          continue;
        }
        if (blk != have) {
          flush();
          have = blk;
        }
        if (flying < S) wait_vm<0>();
        else if (late > 0) wait_vm<(S - 1) * ST2::XI>();
        else wait_vm<(S - 1) * PER2>();
        late -= late > 0;
        asm volatile("" ::: "memory");
        ST2 s;
        s.read(ring_p + tail * SLOT, lane);
        reads_done();
        taken();
        copy_next();
        s.multiply(acc);
        st += W;
      }
      flush();
      lds_barrier();
      store_y(item);
      lds_barrier();
    }
  }
}

// ---------------------------------------------------------------------------

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }
// Parts of d in the logits' partial sums: more of them spread the router's
// weights over more CUs, but every workgroup of the second kernel reads all.
int router_parts(const moe_desc& d) { return d.T <= 4 ? 8 : 2; }
int64_t part_bytes(const moe_desc& d) { return align256((int64_t)router_parts(d) * d.T * d.E * 4); }
constexpr int64_t SYNC_BYTES = 4096;
constexpr int MAX_WGS = SYNC_BYTES / 4 - SYNC_FLAGS;

template <int GRP, int TMAX, int RB, int R1, int R2, int SUB2, int W, int S>
hipError_t run(const DecodeParams& p, int grid, hipStream_t s) {
  decode_kernel<GRP, TMAX, RB, R1, R2, SUB2, W, S><<<(unsigned)grid, 64 * (W + 1), 0, s>>>(p);
  return hipGetLastError();
}

template <int GRP>
hipError_t decode(const DecodeParams& p, int grid, hipStream_t s) {
  if constexpr (GRP == 0) {
    if (p.T <= 2) return run<0, 2, 2, 16, 8, 2, 8, 6>(p, grid, s);
    return run<0, MAX_T, 16, 16, 16, 1, 8, 3>(p, grid, s);
  } else {
    if (p.T <= 2) return run<GRP, 2, 2, 16, 8, 1, 8, 4>(p, grid, s);
    return run<GRP, MAX_T, 16, 32, 16, 1, 4, 2>(p, grid, s);
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
    decode_router_kernel<1><<<rgrid, 256, 0, s>>>((const uint16_t*)x, (const uint16_t*)Wr, d.T, d.d, d.E, part, sync,
                                                  SYNC_FLAGS + grid);
  else
    decode_router_kernel<4><<<rgrid, 256, 0, s>>>((const uint16_t*)x, (const uint16_t*)Wr, d.T, d.d, d.E, part, sync,
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
