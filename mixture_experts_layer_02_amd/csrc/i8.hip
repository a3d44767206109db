// INT8 products with one scale per token and per channel: the row quantiser,
// the kernel for products of few rows, and the choice between it and the
// 256 x 256 tiles of gemm_dma.h.
//
// A row v is held as codes q and one float32 scale s = max|v| / 127, with
// q = 127 v / max|v| rounded to nearest, ties to even; v is about s q.  A
// product of two quantised matrices is then exact in whole numbers up to the
// two scales: <x, w> = s_x s_w <q_x, q_w>, and the 32-bit sums of the int8
// matrix instructions lose nothing (K up to 2^17 at |code| = 127).
#include <algorithm>
#include <type_traits>

#include "gemm_dma.h"
#include "internal.h"

namespace moe {

namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// Row quantiser
// ---------------------------------------------------------------------------

// The 16-byte vector of a row as float: 8 bf16 or 4 float values.
__device__ __forceinline__ void unpack(u32x4_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(u32x4_t w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, WAVE));
  return v;
}

// A row's quantisation from its largest |value| (as bits, so that NaN > inf >
// every number).  The codes are 127 v / max rounded to nearest, ties to even,
// exactly: r = v (127 / max) is off by at most 2^-23 of itself, so the integer
// nearest to r is right unless r lies about that near to a tie (the slow form;
// 2 10^-4 is asked, for |r| up to 127).  There, for float values, the quotient is taken
// in 64 bits, where none is nearer than 2^-40 of itself to a tie without being
// one.  For bf16 values, of 8 bits each, 254 v = (2n + 1) max is an equation of
// whole numbers up to 255^2 and a power of two, so none is nearer than 1.5 10^-5
// of itself: what lies within 10^-6 of itself is a tie (v = max / 2 is: 63.5),
// and the even neighbour is 2 rint(r / 2).  A row of zeros has scale 0; a row
// with an infinity or a NaN has scale NaN and codes 0, so that what is computed
// from it is NaN.
struct RowQuant {
  float top, inv;
  bool small;  // 127 / max overflows: every quotient in 64 bits
  bool none;   // all codes are zero
  __device__ __forceinline__ explicit RowQuant(uint32_t bits) {
    top = __uint_as_float(bits);
    none = bits == 0 || bits >= 0x7f800000u;
    small = !none && top < 0x1p-100f;
    inv = none || small ? 0.f : 127.0f / top;
  }
  __device__ __forceinline__ float scale() const {
    return none && __float_as_uint(top) ? __uint_as_float(0x7fc00000u) : top / 127.0f;
  }
  // N codes, four to a dword.  r + 1.5 2^23 rounds r to the nearest integer,
  // ties to even, in the low bits of its own bit pattern.
  template <bool EXACT, int N>
  __device__ __forceinline__ void codes(const float (&v)[N], uint32_t (&o)[(N + 3) / 4]) const {
    constexpr float MAGIC = 12582912.0f;
    uint32_t b[N];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r = none ? 0.f : v[i] * inv;
      const float m = r + MAGIC;
      b[i] = __float_as_uint(m);
      off = fmaxf(off, fabsf(r - (m - MAGIC)));
    }
    if (off > 0.4998f || small) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float r = v[i] * inv;
        const bool tie = fabsf(fabsf(r - truncf(r)) - 0.5f) < 1e-6f * fabsf(r);
        int q = (int)rintf(r);
        if (EXACT ? tie || small : small) q = (int)rint((double)v[i] * 127.0 / (double)top);
        else if (tie) q = 2 * (int)rintf(r * 0.5f);
        b[i] = (uint32_t)q;
      }
    }
#pragma unroll
    for (int j = 0; j < (N + 3) / 4; ++j) {
      o[j] = 0;
#pragma unroll
      for (int i = 4 * j; i < N && i < 4 * j + 4; ++i) o[j] |= (b[i] & 0xffu) << (8 * (i - 4 * j));
    }
  }
};

// W waves per row.  NV > 0: the row is held in NV vectors per lane and read
// once; NV = 0: any length, read twice (the second time from cache).  VEC:
// rows start at multiples of 16 bytes, so values and codes go as vectors,
// through buffer resources that end with the row (loads past it give zeros,
// stores past it are dropped, each by whole 4 bytes).  nrows (device, or NULL):
// rows at or past it are left alone.
// Bound by HBM, (b + 1) bytes a value; with few rows by one row's latency,
// hence four waves on it.
template <typename T, int W, int NV, bool VEC>
__global__ void __launch_bounds__(256) i8_quant_rows_kernel(const T* __restrict__ w, int64_t rows, int cols,
                                                            int64_t ldw, const int32_t* __restrict__ nrows,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
  constexpr int N = VEC ? 16 / sizeof(T) : 1;  // values per load
  constexpr int L = W * 64;                    // lanes per row
  constexpr bool EXACT = sizeof(T) == 4;
  __shared__ uint32_t s_top[4];
  const int sub = threadIdx.x % L;
  const int rw = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int64_t lim = nrows ? min(rows, (int64_t)max(*nrows, 0)) : rows;
  for (int64_t r = (int64_t)blockIdx.x * (4 / W) + rw; r < lim; r += (int64_t)gridDim.x * (4 / W)) {
    T* src = const_cast<T*>(w) + r * ldw;
    int8_t* dst = q + r * ldq;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(src, (short)0, (int)((cols * sizeof(T) + 3) & ~3u), 0x00020000);
    const __amdgpu_buffer_rsrc_t rd = __builtin_amdgcn_make_buffer_rsrc(dst, (short)0, cols & ~3, 0x00020000);
    // The N values of column c and on, as they lie in memory.
    using Raw = typename std::conditional<VEC, u32x4_t, float>::type;
    auto load = [&](int c) -> Raw {
      if constexpr (VEC) {
        u32x4_t x = __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)c * (uint32_t)sizeof(T), 0, 0);
        if (sizeof(T) == 2 && (cols & 1) && c < cols && c + N > cols) {  // half of the row's last 4 bytes is not its own
          const int d = (cols - c) >> 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] &= i == d ? 0xffffu : 0xffffffffu;
        }
        return x;
      } else {
        return Elem<T>::ld(src, c);
      }
    };
    auto wide = [&](const Raw& x, float (&v)[N]) {
      if constexpr (VEC) unpack(x, v);
      else v[0] = x;
    };
    uint32_t top = 0;
    auto grow = [&](const Raw& x) {
      float v[N];
      wide(x, v);
#pragma unroll
      for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    };
    Raw held[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) held[j] = load((j * L + sub) * N);
#pragma unroll
      for (int j = 0; j < NV; ++j) grow(held[j]);
    } else {
      for (int c = sub * N; c < cols; c += L * N) grow(load(c));
    }
    top = wave_max(top);
    if constexpr (W > 1) {  // (every wave of the workgroup has the same row)
      __syncthreads();
      if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) top = max(top, s_top[i]);
    }
    const RowQuant rq(top);
    auto put = [&](int c, const Raw& x) {
      float v[N];
      wide(x, v);
      uint32_t o[(N + 3) / 4];
      rq.template codes<EXACT, N>(v, o);
      if constexpr (!VEC) {
        dst[c] = (int8_t)o[0];
      } else {
        if constexpr (N == 8) __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{o[0], o[1]}, rd, (uint32_t)c, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(o[0], rd, (uint32_t)c, 0, 0);
        if ((cols & 3) && c < cols && c + N > (cols & ~3)) {  // the row's last one to three codes
          const int z = cols & ~3;
          for (int i = z; i < cols; ++i) dst[i] = (int8_t)(o[(z - c) / 4] >> (8 * (i - z)));
        }
      }
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (VEC) asm volatile("" : "+v"(held[j]));  // widened again, not kept as float
        put((j * L + sub) * N, held[j]);
      }
    } else {
      for (int c = sub * N; c < cols; c += L * N) put(c, load(c));
    }
    if (sub == 0) scale[r] = rq.scale();
  }
}

template <typename T>
hipError_t quant_rows(const T* w, int64_t rows, int cols, int64_t ldw, const int32_t* nrows, int8_t* q,
                      int64_t ldq, float* scale, hipStream_t s) {
  constexpr int64_t N = 16 / sizeof(T);
  const int64_t nv = cdiv(cols, 64 * N);  // vectors per lane of one wave
  const int64_t cap = (int64_t)num_cus() * 16;
  const bool vec = ldw % N == 0;
  // Short rows, many of them: a wave each (16384 x 1792 bf16: 20 us, 4.5 TB/s;
  // a workgroup each: 37 us).  Else a workgroup per row (16384 x 6144 bf16: 61
  // us, 5.0 TB/s; a wave each: 73 us; one row of 6144: 4.3 against 6.2 us).
  if (vec && nv <= 4 && rows >= 1024) {
    const unsigned grid = (unsigned)std::min(cdiv(rows, 4), cap);
    i8_quant_rows_kernel<T, 1, 4, true><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)std::min(rows, cap);
  if (!vec) i8_quant_rows_kernel<T, 4, 0, false><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale);
  else if (nv <= 12) i8_quant_rows_kernel<T, 4, 3, true><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale);
  else if (nv <= 32) i8_quant_rows_kernel<T, 4, 8, true><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale);
  else i8_quant_rows_kernel<T, 4, 0, true><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Products of few rows
// ---------------------------------------------------------------------------

// y[r][n] = sx[r] sw[n] <x[r], w[n]> for the rows of every group g (expert),
// r in [offsets[g], offsets[g+1]), w the group's [N][K] codes.  offsets NULL:
// one group of M rows.  DUAL: two weights, y = silu(G) U and, when gu is set,
// G and U.  row_token set: x[r] and sx[r] are those of row row_token[r].
struct I8Params {
  const int8_t* x;
  int64_t ldx;
  const float* sx;
  const int32_t* row_token;
  int64_t x_rows;  // rows of x behind row_token
  const int8_t* w;
  const int8_t* w2;
  int64_t ldw;
  const float* sw;
  const float* sw2;
  const float* bias;
  const int32_t* offsets;
  int ngroups;
  int M, N, K;
  int64_t tiles;  // workgroups' worth of work: m-tile slots times channel tiles
  int by_slot;    // how these go to the XCDs (see tile_of)
  void* y;
  int64_t ldy;
  uint16_t* gu;
};

// The group and the rows [m0, m0 + mlim) of m-tile `slot`: groups have
// ceil(rows / MT) m-tiles each, in order.  Every wave searches alike, 64 groups
// at a time.  False past the last m-tile.
template <int MT>
__device__ __forceinline__ bool find_tile(const I8Params& p, int slot, int lane, int& g, int& m0, int& mlim) {
  g = 0;
  m0 = slot * MT;
  int m1 = p.M;
  if (!p.offsets && m0 >= m1) g = -1;
  if (p.offsets) {
    int before = 0;
    g = -1;
    for (int base = 0; base < p.ngroups; base += 64) {
      const int i = base + lane;
      const int lo = i < p.ngroups ? p.offsets[i] : 0, hi = i < p.ngroups ? p.offsets[i + 1] : 0;
      const int c = (hi - lo + MT - 1) / MT;
      int inc = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(inc, o, WAVE);
        if (lane >= o) inc += v;
      }
      const unsigned long long past = __ballot(before + inc > slot);
      if (past) {
        const int l = __ffsll(past) - 1;
        g = base + l;
        m0 = __shfl(lo, l, WAVE) + (slot - before - (__shfl(inc, l, WAVE) - __shfl(c, l, WAVE))) * MT;
        m1 = __shfl(hi, l, WAVE);
        break;
      }
      before += __shfl(inc, 63, WAVE);
    }
  }
  g = __builtin_amdgcn_readfirstlane(g);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  mlim = __builtin_amdgcn_readfirstlane(min(MT, m1 - m0));
  return g >= 0;
}

// The scales (or biases) of channels n .. n + 3 of a row of N at `base`, n a
// multiple of 4; zeros past N.
__device__ __forceinline__ f32x4_t load4(const float* base, int n, int N) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (N % 4 == 0) {  // (then rows start at multiples of 16 bytes, and the four are all inside or all outside)
    if (n < N) v = *reinterpret_cast<const f32x4_t*>(base + n);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < N) v[q] = base[n + q];
  }
  return v;
}

// The scales and bias of a lane's four channels, loaded ahead of their use.
struct Channels {
  f32x4_t s1, s2, b;  // of the weight (DUAL: the gate's and the up's); the bias
  template <bool DUAL>
  __device__ __forceinline__ void load(const I8Params& p, int g, int n) {
    s1 = load4(p.sw + (int64_t)g * p.N, n, p.N);
    if (DUAL) s2 = load4(p.sw2 + (int64_t)g * p.N, n, p.N);
    else b = p.bias ? load4(p.bias, n, p.N) : f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
};

// Tile `id` (XCD id mod 8) of a product with ntiles channel tiles: its m-tile
// slot and channel tile (which may be past the last).  by_slot: an m-tile's
// channel tiles are all on one XCD, one after the other, so its L2 holds the
// rows of the few m-tiles in work there.  Else the channel tile fixes the XCD,
// whose L2 then serves a weight tile to all the m-tiles that share it.
__device__ __forceinline__ void tile_of(const I8Params& p, int64_t id, int ntiles, int& slot, int& ntile) {
  const int x = (int)(id & 7);
  const int64_t j = id >> 3;
  if (p.by_slot) {
    slot = (int)(j / ntiles) * 8 + x;
    ntile = (int)(j % ntiles);
  } else {
    const int per = (ntiles + 7) >> 3;
    slot = (int)(j / per);
    ntile = (int)(j % per) * 8 + x;
  }
}
int64_t tile_count(const I8Params& p, int64_t slots, int64_t ntiles) {
  return p.by_slot ? cdiv(slots, 8) * 8 * ntiles : slots * cdiv(ntiles, 8) * 8;
}

// The outputs of one row r at channels n .. n + 3 (n < N) from their sums: s1
// alone, or gate s1 and up s2.
template <bool DUAL, typename OUT>
__device__ __forceinline__ void store4(const I8Params& p, int64_t r, int n, float sx, const Channels& ch, i32x4_t s1,
                                       i32x4_t s2) {
  float o[4];
  if constexpr (DUAL) {
    float gt[4], up[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // (N is a multiple of 64)
      gt[q] = (float)s1[q] * sx * ch.s1[q];
      up[q] = (float)s2[q] * sx * ch.s2[q];
      o[q] = gt[q] * sigmoidf_(gt[q]) * up[q];
    }
    if (p.gu) {
      uint16_t* gr = p.gu + r * 2 * p.N + n;
      *reinterpret_cast<u32x2_t*>(gr) = u32x2_t{pack_bf2(gt[0], gt[1]), pack_bf2(gt[2], gt[3])};
      *reinterpret_cast<u32x2_t*>(gr + p.N) = u32x2_t{pack_bf2(up[0], up[1]), pack_bf2(up[2], up[3])};
    }
  } else {
    // (the product rounded before the bias is added, here and in gemm_dma.h's
    // epilogue: a row's outputs are the same whichever kernel takes it)
#pragma clang fp contract(off)
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = (float)s1[q] * sx * ch.s1[q] + ch.b[q];
  }
  OUT* y = reinterpret_cast<OUT*>(p.y) + r * p.ldy + n;
  if (p.N % 4 == 0 && p.ldy % 4 == 0) {  // (then the four are inside and their address is aligned)
    if constexpr (sizeof(OUT) == 2)
      *reinterpret_cast<u32x2_t*>(y) = u32x2_t{pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3])};
    else *reinterpret_cast<f32x4_t*>(y) = f32x4_t{o[0], o[1], o[2], o[3]};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < p.N) Elem<OUT>::st(y, q, o[q]);
  }
}

// LDS rows are 128 bytes; the 16-byte piece c of row r sits at c ^ swz16(r).  A
// ds_read_b128 goes by groups of 16 lanes (0-3, 12-15, 20-23, 24-27, the rest
// of the first 32, and likewise the second), and a fragment's lane l reads
// piece c + l / 16 of row l % 16: with this swizzle a group's 16 pieces are
// spread over all 64 banks (none of the reads conflicts; with gemm_dma.h's,
// made for 32 rows of one piece, half of the read cycles did).
__device__ __forceinline__ int swz16(int r) { return r & 6; }

// Zeroes the codes at k >= K of a fragment whose lane holds 16 codes from k on.
__device__ __forceinline__ i32x4_t mask_k(i32x4_t f, int left) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int v = left - 4 * d;
    f[d] &= v >= 4 ? -1 : v <= 0 ? 0 : (int)((1u << (8 * v)) - 1u);
  }
  return f;
}

// With few rows the product streams the weights, each of whose bytes is used
// by one workgroup only: the kernel is bound by HBM and has to keep many loads
// in flight.  A workgroup computes MB*16 rows x NB*16 channels (DUAL: half of
// them gate, half up) over all of K, cut into chunks of 128 codes that its
// W waves take in turn; no wave shares an operand with another, so the main
// loop has no barrier: each wave copies a chunk into its own part of LDS (LDS
// DMA, 8 rows x 128 bytes per instruction, all lines whole), waits for it,
// takes it to registers, starts the next copy over it and multiplies.  Several
// workgroups share a CU (at least WPS waves per SIMD), so a CU's whole LDS is in
// flight most of the time.  (Measured on gate/up, d = 6144, f = 1792, 96 experts
// of which 21 rows each: 372 us, 5.7 TB/s; a ring of two stages with half the
// workgroups took 512 us, chunks of 64 codes, half lines, 451 us.)  The W partial
// sums are whole numbers and are added through LDS at the end, in any order with
// the same result.
//   Fragments: v_mfma_i32_16x16x64_i8 with the channels as rows and the tokens
//   as columns; lane l holds 16 codes of row l % 16 at k = 16 (l / 16), and
//   the result's rows 4 (l / 16) .. + 3 of column l % 16, so a lane's four
//   sums are consecutive channels of one token.
//   LDS: rows of 128 bytes, 16-byte piece c of row r at c ^ swz16(r).
template <int MB, int NB, int W, int WPS, bool DUAL, typename OUT>
__global__ void __launch_bounds__(64 * W, WPS) i8_few_rows_kernel(I8Params p) {
  using namespace dma;
  static_assert(!DUAL || NB % 2 == 0, "gate and up blocks");
  constexpr int MT = MB * 16, NT = NB * 16;
  constexpr int OC = DUAL ? NT / 2 : NT;       // output channels
  constexpr int STAGE = (MT + NT) * 128;       // bytes: weight rows, then token rows
  constexpr int PER = (MT + NT) / 8;           // copies per chunk
  constexpr int RP = NT + 4;                   // pitch of the partial sums (ints)
  constexpr int RING = W * STAGE, RED = W * MT * RP * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > RED ? RING : RED];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntiles = (p.N + OC - 1) / OC;
  for (int64_t id = blockIdx.x; id < p.tiles; id += gridDim.x) {
    int slot, ntile;
    tile_of(p, id, ntiles, slot, ntile);
    if (ntile >= ntiles) continue;

    int g, m0, mlim;
    if (!find_tile<MT>(p, slot, lane, g, m0, mlim)) break;  // (every later slot is past the last m-tile too)
    const int n0 = ntile * OC, nlim = min(OC, p.N - n0);

    // Copy offsets.  Copy j moves LDS rows 8j .. 8j + 7: lane i row 8j + i/8,
    // position i % 8, which holds piece (i % 8) ^ swz_k(row) of the row's 128
    // bytes.  Rows that do not exist get bit 31, past every resource: zeros.
    const i32x4 rw = make_rsrc(p.w + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw);
    const i32x4 rw2 = DUAL ? make_rsrc(p.w2 + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw) : rw;
    const i32x4 rx = p.row_token ? make_rsrc(p.x, (uint64_t)p.x_rows * p.ldx)
                                 : make_rsrc(p.x + (int64_t)m0 * p.ldx, (uint64_t)mlim * p.ldx);
    uint32_t vw[NT / 8], vx[MT / 8];
    auto piece = [&](int row) { return (lane & 7) ^ swz16(row); };
#pragma unroll
    for (int j = 0; j < NT / 8; ++j) {
      const int row = 8 * j + (lane >> 3), src = DUAL && row >= OC ? row - OC : row;
      vw[j] = src < nlim ? (uint32_t)(src * p.ldw) + piece(row) * 16 : 0x80000000u;
    }
#pragma unroll
    for (int j = 0; j < MT / 8; ++j) {
      const int row = 8 * j + (lane >> 3);
      uint32_t src = row;
      if (p.row_token && row < mlim) src = p.row_token[m0 + row];
      vx[j] = row < mlim ? (uint32_t)(src * p.ldx) + piece(row) * 16 : 0x80000000u;
    }

    const int chunks = (p.K + 127) / 128;
    const int mine = (chunks - wave + W - 1) / W;  // chunks wave, wave + W, ...
    const uint32_t st_lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem) + wave * STAGE;
    const uint8_t* st = smem + wave * STAGE;
    auto k_of = [&](int i) { return (wave + W * i) * 128; };
    // The wave's chunk i.  TAIL: it is K's last and not whole: a piece past K
    // lies in the next row, and none of it is wanted.
    auto copy_as = [&](int k0, auto tail_c) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const bool tok = j >= NT / 8;
        const int jj = tok ? j - NT / 8 : j;
        uint32_t v = tok ? vx[tok ? jj : 0] : vw[tok ? 0 : jj];
        if (decltype(tail_c)::value && k0 + piece(8 * jj + (lane >> 3)) * 16 >= p.K) v = 0x80000000u;
        const i32x4 r = tok ? rx : (DUAL && j >= NT / 16 ? rw2 : rw);
        dma16(r, v, (uint32_t)k0, __builtin_amdgcn_readfirstlane(st_lds + j * 1024));
      }
    };
    auto copy = [&](int i) {
      const int k0 = k_of(i);
      if (k0 + 128 <= p.K) copy_as(k0, std::false_type());
      else copy_as(k0, std::true_type());
    };

    i32x4_t acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};

    // The epilogue's scales, asked for now: thread tid has the channels c_out ..
    // + 3 of rows tid / VPR, + RPI, ...
    constexpr int VPR = OC / 4, RPI = 64 * W / VPR, IT = (MT + RPI - 1) / RPI;
    const int c_out = (tid % VPR) * 4;
    Channels ch;
    ch.template load<DUAL>(p, g, n0 + c_out);
    float sx[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int row = tid / VPR + i * RPI;
      sx[i] = row < mlim ? p.sx[p.row_token ? p.row_token[m0 + row] : m0 + row] : 0.f;
    }

    // A chunk to registers, the next one's copies, its products.
    auto step = [&](int i, auto tail_c) {
      wait_vm<0>();
      asm volatile("" ::: "memory");
      i32x4_t fw[2][NB], fx[2][MB];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int r = b * 16 + (lane & 15);
          fx[ks][b] = *reinterpret_cast<const i32x4_t*>(st + (NT + r) * 128 +
                                                         (((4 * ks + (lane >> 4)) ^ swz16(r)) << 4));
        }
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const int r = a * 16 + (lane & 15);
          fw[ks][a] = *reinterpret_cast<const i32x4_t*>(st + r * 128 + (((4 * ks + (lane >> 4)) ^ swz16(r)) << 4));
        }
      }
      // The chunk is in registers before the next one is copied over it.
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      asm volatile("" ::: "memory");
      if (i + 1 < mine) copy(i + 1);
      if constexpr (decltype(tail_c)::value) {
        // the codes past K in the row's last piece are not the caller's to give:
        // zeroed in one operand, the other's do not matter
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int b = 0; b < MB; ++b) fx[ks][b] = mask_k(fx[ks][b], p.K - (k_of(i) + ks * 64 + (lane >> 4) * 16));
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int a = 0; a < NB; ++a)
#pragma unroll
          for (int b = 0; b < MB; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[ks][a], fx[ks][b], acc[a][b], 0, 0, 0);
    };
    const bool tail = p.K % 16 && mine > 0 && k_of(mine - 1) + 128 > p.K;  // the wave's last chunk needs the mask
    const int plain = tail ? mine - 1 : mine;
    if (mine > 0) copy(0);
    for (int i = 0; i < plain; ++i) step(i, std::false_type());
    if (tail) step(plain, std::true_type());

    // Partial sums [wave][token][channel] over the ring, once every wave is done with it.
    __syncthreads();
    int* red = reinterpret_cast<int*>(smem);
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b)
        *reinterpret_cast<i32x4_t*>(red + (wave * MT + b * 16 + (lane & 15)) * RP + a * 16 + (lane >> 4) * 4) = acc[a][b];
    __syncthreads();
    auto total = [&](int row, int c) {
      i32x4_t v = *reinterpret_cast<const i32x4_t*>(red + row * RP + c);
#pragma unroll
      for (int w = 1; w < W; ++w) v += *reinterpret_cast<const i32x4_t*>(red + (w * MT + row) * RP + c);
      return v;
    };
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int row = tid / VPR + i * RPI;
      if (row < mlim && c_out < nlim) {
        const i32x4_t s1 = total(row, c_out);
        store4<DUAL, OUT>(p, (int64_t)m0 + row, n0 + c_out, sx[i], ch, s1, DUAL ? total(row, OC + c_out) : s1);
      }
    }
    __syncthreads();  // the next tile's copies overwrite the partial sums
  }
}

// Between those and the tiles of gemm_dma.h: MT rows x NT channels (DUAL: half
// of them gate, half up), whose operands WM x WN waves share in LDS, in chunks
// of 128 codes of k; a wave has MT / WM rows and NT / WN channels.  Swizzle and
// fragments as above.  The tokens of a chunk, which come from the cache, are
// copied one chunk ahead, its weights, which come from HBM, SW - 1 chunks (128
// x 128, gate/up of 96 experts, 63 rows each: SW = 2 428 us, SW = 3 408).  Small
// tiles have two or three workgroups on a CU, so one's waits, barriers and
// epilogue pass under the others' copies; the largest fills the CU's LDS with
// one workgroup of eight waves, which copies least per product.  Blocks of 16
// rows that the m-tile does not have are left out: the loop is built for each
// number of them (in steps of a quarter), so that it has no branch and reads all
// its fragments before it multiplies (with branches and one fragment at a time
// linear 1000 x 6144 x 1792 took 27 us, now 21-23), and tokens that are not there
// are not copied.  Rows are copied half as often per weight as by the kernel
// above: gate/up of 96 experts, 43 rows each, 387 against 433 us.
template <int MT, int NT, int WM, int WN, int WGS, int SW, bool DUAL, typename OUT>
__global__ void __launch_bounds__(64 * WM * WN, WGS) i8_mid_rows_kernel(I8Params p) {
  using namespace dma;
  constexpr int OC = DUAL ? NT / 2 : NT, W = WM * WN;
  constexpr int MB = MT / WM / 16, NB = NT / WN / 16;  // a wave's blocks of 16 rows and 16 channels
  constexpr int WST = NT * 128, XST = MT * 128;        // bytes of a chunk: weight rows, token rows
  constexpr int CW = NT / 8 / W, CX = MT / 8 / W;      // copies per wave and chunk: of weight rows, of token rows
  constexpr int KB = NB * MB > 16 ? 1 : 2;             // k-steps whose fragments are read at once
  constexpr bool PIPE = DUAL && WGS == 1;               // (see pipe)
  static_assert(!PIPE || (SW > 2 && NB % 4 == 0), "stages and halves of pipe");
  static_assert(CW * 8 * W == NT && CX * 8 * W == MT, "shares of the copies");
  static_assert(!DUAL || (CW % 4 == 0 && NB % 2 == 0), "gate and up blocks");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SW * WST + 2 * XST];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int ntiles = (p.N + OC - 1) / OC;
  for (int64_t id = blockIdx.x; id < p.tiles; id += gridDim.x) {
    int slot, ntile, g, m0, mlim;
    tile_of(p, id, ntiles, slot, ntile);
    if (ntile >= ntiles) continue;
    if (!find_tile<MT>(p, slot, lane, g, m0, mlim)) break;
    const int n0 = ntile * OC, nlim = min(OC, p.N - n0);
    const i32x4 rw = make_rsrc(p.w + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw);
    const i32x4 rw2 = DUAL ? make_rsrc(p.w2 + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw) : rw;
    const i32x4 rx = p.row_token ? make_rsrc(p.x, (uint64_t)p.x_rows * p.ldx)
                                 : make_rsrc(p.x + (int64_t)m0 * p.ldx, (uint64_t)mlim * p.ldx);
    // A wave copies CW times 8 of the weight rows, and of the token rows every
    // W-th eight.  With DUAL a wave's channel blocks are gate, up, gate, up ..:
    // LDS weight row r is gate or up by bit 4, channel 16 (r / 32) + r % 16.
    uint32_t vw[CW], vx[CX];
    auto row_w = [&](int j) { return 8 * (wave * CW + j); };
    auto row_x = [&](int j) { return 8 * (wave + W * j); };
    auto piece = [&](int row8) { return ((lane & 7) ^ swz16(row8 + (lane >> 3))) << 4; };
#pragma unroll
    for (int j = 0; j < CW; ++j) {
      const int row = row_w(j) + (lane >> 3), src = DUAL ? (row >> 5) * 16 + (row & 15) : row;
      vw[j] = src < nlim ? (uint32_t)(src * p.ldw) + piece(row_w(j)) : 0x80000000u;
    }
#pragma unroll
    for (int j = 0; j < CX; ++j) {
      const int row = row_x(j) + (lane >> 3);
      uint32_t src = row;
      if (p.row_token && row < mlim) src = p.row_token[m0 + row];
      vx[j] = row < mlim ? (uint32_t)(src * p.ldx) + piece(row_x(j)) : 0x80000000u;
    }
    const int chunks = (p.K + 127) / 128;
    const uint32_t lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
    // Chunk i's weights to ring stage i % SW, its tokens to i % 2 (TAIL as
    // above).  Eights of token rows that the m-tile does not have are left as
    // they are: nothing is stored of their products.
    auto copy_w_as = [&](int i, auto tail_c) {
      const uint32_t st = lds + (uint32_t)(i % SW) * WST;
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        uint32_t o = vw[j];
        if (decltype(tail_c)::value && i * 128 + piece(row_w(j)) >= p.K) o = 0x80000000u;
        const i32x4 r = DUAL && (j & 2) ? rw2 : rw;  // (bit 4 of an LDS weight row: gate or up)
        dma16(r, o, (uint32_t)(i * 128), __builtin_amdgcn_readfirstlane(st + row_w(j) * 128));
      }
    };
    auto copy_x_as = [&](int i, auto tail_c) {
      const uint32_t st = lds + SW * WST + (uint32_t)(i & 1) * XST;
#pragma unroll
      for (int j = 0; j < CX; ++j) {
        if (row_x(j) >= mlim) break;
        uint32_t o = vx[j];
        if (decltype(tail_c)::value && i * 128 + piece(row_x(j)) >= p.K) o = 0x80000000u;
        dma16(rx, o, (uint32_t)(i * 128), __builtin_amdgcn_readfirstlane(st + row_x(j) * 128));
      }
    };
    auto copy_w = [&](int i) {
      if (i * 128 + 128 <= p.K) copy_w_as(i, std::false_type());
      else if (i < chunks) copy_w_as(i, std::true_type());
    };
    auto copy_x = [&](int i) {
      if (i * 128 + 128 <= p.K) copy_x_as(i, std::false_type());
      else if (i < chunks) copy_x_as(i, std::true_type());
    };

    // The tile's row blocks go to the wave rows in turn; a wave's that exist:
    const int blocks = ((mlim + 15) / 16 - wm + WM - 1) / WM;
    i32x4_t acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};

    // The epilogue's scales, asked for now.
    constexpr int AS = DUAL ? 2 : 1;  // weight blocks of an output block
    auto c_out = [&](int a) { return (wn * NB + a) * (DUAL ? 8 : 16) + (lane >> 4) * 4; };
    Channels ch[NB / AS];
    float sx[MB];
    auto scales = [&]() {
#pragma unroll
      for (int a = 0; a < NB; a += AS) ch[a / AS].template load<DUAL>(p, g, n0 + c_out(a));
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const int row = (b * WM + wm) * 16 + (lane & 15);
        sx[b] = row < mlim ? p.sx[p.row_token ? p.row_token[m0 + row] : m0 + row] : 0.f;
      }
    };
    if (!PIPE) scales();

    // Chunk i: the next one's copies, its fragments, its products with the
    // first MBA row blocks.
    auto step = [&](int i, auto mba_c, auto tail_c) {
      constexpr int MBA = decltype(mba_c)::value;
      // (the last copies asked for, the weights of chunk i + SW - 2, may be on their way still)
      if (SW > 2 && i + SW - 2 < chunks) wait_vm<CW>();
      else wait_vm<0>();
      lds_barrier();  // chunk i has landed for every wave, and every wave has read chunk i - 1
      copy_x(i + 1);
      copy_w(i + SW - 1);
      const uint8_t* st = smem + (uint32_t)(i % SW) * WST;
      const uint8_t* stx = smem + SW * WST + (i & 1) * XST;
#pragma unroll
      for (int k = 0; k < 2; k += KB) {
        i32x4_t fw[KB][NB], fx[KB][MBA > 0 ? MBA : 1];
#pragma unroll
        for (int kk = 0; kk < KB; ++kk) {
          const int ks = k + kk;
#pragma unroll
          for (int a = 0; a < (MBA > 0 ? NB : 0); ++a) {
            const int r = (wn * NB + a) * 16 + (lane & 15);
            fw[kk][a] = *reinterpret_cast<const i32x4_t*>(st + r * 128 + (((4 * ks + (lane >> 4)) ^ swz16(r)) << 4));
            if constexpr (decltype(tail_c)::value)
              fw[kk][a] = mask_k(fw[kk][a], p.K - (i * 128 + ks * 64 + (lane >> 4) * 16));
          }
#pragma unroll
          for (int b = 0; b < MBA; ++b) {
            const int r = (b * WM + wm) * 16 + (lane & 15);
            fx[kk][b] = *reinterpret_cast<const i32x4_t*>(stx + r * 128 + (((4 * ks + (lane >> 4)) ^ swz16(r)) << 4));
          }
        }
#pragma unroll
        for (int kk = 0; kk < KB; ++kk)
#pragma unroll
          for (int b = 0; b < MBA; ++b)
#pragma unroll
            for (int a = 0; a < NB; ++a)
              acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[kk][a], fx[kk][b], acc[a][b], 0, 0, 0);
      }
    };
    // PIPE: one workgroup on the CU, so its fragments are read while it
    // multiplies: a chunk goes in four parts, by k-step and half of the channel
    // blocks, and each part's products pass under the next part's reads, the
    // last one's under the next chunk's, so the barrier between chunks lies
    // before the last part: there every wave has read the whole chunk, and the
    // copies into its stages start.
    auto pipe = [&](auto mba_c) {
      constexpr int MBA = decltype(mba_c)::value, M1 = MBA > 0 ? MBA : 1, HB = MBA > 0 ? NB / 2 : 0;
      i32x4_t x0[M1], x1[M1], wa[NB / 2], wb[NB / 2];
      auto at = [&](const uint8_t* s, int r, int ks) {
        return *reinterpret_cast<const i32x4_t*>(s + r * 128 + (((4 * ks + (lane >> 4)) ^ swz16(r)) << 4));
      };
      auto read_x = [&](i32x4_t (&f)[M1], int i, int ks) {
        const uint8_t* s = smem + SW * WST + (i & 1) * XST;
#pragma unroll
        for (int b = 0; b < MBA; ++b) f[b] = at(s, (b * WM + wm) * 16 + (lane & 15), ks);
      };
      auto read_w = [&](i32x4_t (&f)[NB / 2], int i, int ks, int half) {
        const uint8_t* s = smem + (uint32_t)(i % SW) * WST;
#pragma unroll
        for (int a = 0; a < HB; ++a) f[a] = at(s, (wn * NB + half * (NB / 2) + a) * 16 + (lane & 15), ks);
      };
      auto mul = [&](const i32x4_t (&w)[NB / 2], const i32x4_t (&x)[M1], auto half_c) {
        constexpr int A0 = decltype(half_c)::value * (NB / 2);
#pragma unroll
        for (int a = 0; a < HB; ++a)
#pragma unroll
          for (int b = 0; b < MBA; ++b)
            acc[A0 + a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[a], x[b], acc[A0 + a][b], 0, 0, 0);
      };
      const std::integral_constant<int, 0> h0;
      const std::integral_constant<int, 1> h1;
      read_x(x0, 0, 0);
      read_w(wa, 0, 0, 0);
      for (int i = 0; i < chunks; ++i) {
        read_w(wb, i, 0, 1);
        mul(wa, x0, h0);
        read_x(x1, i, 1);
        read_w(wa, i, 1, 0);
        mul(wb, x0, h1);
        read_w(wb, i, 1, 1);
        mul(wa, x1, h0);
        if (i + 1 < chunks) {
          // (the last copies asked for, the weights of chunk i + SW - 1, may be on their way still)
          if (i + SW - 1 < chunks) wait_vm<CW>();
          else wait_vm<0>();
          lds_barrier();  // chunk i + 1 has landed for every wave, and every wave has read chunk i
          copy_x(i + 2);
          copy_w(i + SW);
          read_x(x0, i + 1, 0);
          read_w(wa, i + 1, 0, 0);
        }
        mul(wb, x1, h1);
      }
    };
    const bool tail = p.K % 16 != 0;  // the last chunk needs the mask
    const int plain = tail ? chunks - 1 : chunks;
    auto loop = [&](auto mba_c) {
      if constexpr (PIPE) return pipe(mba_c);
      for (int i = 0; i < plain; ++i) step(i, mba_c, std::false_type());
      if (tail) step(plain, mba_c, std::true_type());
    };
    if constexpr (PIPE) {
      copy_x(0);
      copy_x(1);
#pragma unroll
      for (int i = 0; i < SW; ++i) copy_w(i);
      if (SW <= chunks) wait_vm<(SW - 1) * CW>();
      else wait_vm<0>();
      lds_barrier();
    } else {
      copy_w(0);
      copy_x(0);
#pragma unroll
      for (int i = 1; i < SW - 1; ++i) copy_w(i);
    }
    constexpr int Q = (MB + 3) / 4;  // a loop for each number of row blocks, in steps of a quarter of all
    switch ((blocks + Q - 1) / Q) {
      case 0: loop(std::integral_constant<int, 0>()); break;
      case 1: loop(std::integral_constant<int, Q>()); break;
      case 2: loop(std::integral_constant<int, MB < 2 * Q ? MB : 2 * Q>()); break;
      case 3: loop(std::integral_constant<int, MB < 3 * Q ? MB : 3 * Q>()); break;
      default: loop(std::integral_constant<int, MB>()); break;
    }
    if (PIPE) scales();
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int row = (b * WM + wm) * 16 + (lane & 15);
      if (row >= mlim) continue;
#pragma unroll
      for (int a = 0; a < NB; a += AS)
        if (c_out(a) < nlim)
          store4<DUAL, OUT>(p, (int64_t)m0 + row, n0 + c_out(a), sx[b], ch[a / AS], acc[a][b], acc[a + AS - 1][b]);
    }
    lds_barrier();  // every wave has read the last chunk before the next tile's copies
  }
}

template <int MT, int NT, int WM, int WN, int WGS, int SW, bool DUAL, typename OUT>
hipError_t run_mid(I8Params p, int64_t rows, int64_t groups, int64_t mean, hipStream_t s) {
  // One m-tile per group: nothing shares its weights, so its rows are kept
  // together (gate/up, 105 rows each: 476 us against 515 by channel tiles).
  p.by_slot = p.offsets && groups >= 32 && mean <= MT - MT / 16;
  const int64_t slots = p.offsets ? rows / MT + std::min<int64_t>(p.ngroups, rows) : cdiv(rows, MT);
  p.tiles = tile_count(p, slots, cdiv(p.N, DUAL ? NT / 2 : NT));
  const unsigned grid = (unsigned)std::min<int64_t>(p.tiles, 1 << 22);
  i8_mid_rows_kernel<MT, NT, WM, WN, WGS, SW, DUAL, OUT><<<grid, 64 * WM * WN, 0, s>>>(p);
  return hipGetLastError();
}

template <int MB, int NB, int W, int WPS, bool DUAL, typename OUT>
hipError_t run_few(I8Params p, int64_t rows, hipStream_t s) {
  constexpr int OC = NB * 16 / (DUAL ? 2 : 1);
  // m-tiles at most: every group may end in a partial one
  const int64_t slots = p.offsets ? rows / (MB * 16) + std::min<int64_t>(p.ngroups, rows) : cdiv(rows, MB * 16);
  p.tiles = tile_count(p, slots, cdiv(p.N, OC));
  const unsigned grid = (unsigned)std::min<int64_t>(p.tiles, 1 << 22);  // (a launch has fewer than 2^32 threads)
  i8_few_rows_kernel<MB, NB, W, WPS, DUAL, OUT><<<grid, 64 * W, 0, s>>>(p);
  return hipGetLastError();
}

// The kernel and tile by size.  rows: an upper bound of all rows; groups, mean:
// the groups that have rows and the rows of one of them, as expected from
// evenly spread routing (a skewed one is computed as well, in more m-tiles).
// Times of gate/up of 96 experts, K = 6144, N = 2 x 1792, unless said otherwise.
//   - From 33 rows on the shared-operand kernel, where its tiles fill the chip:
//     64 rows a tile up to 48 (43 rows each: 392 us; 128 rows a tile 398) or
//     where 128 would be too few (linear 2000 x 2048 x 2048, 256 tiles of 128:
//     21.6 us, 64 rows 17.6), else 128 (63 rows: 408 us; 64 rows a tile 484).
//   - Where one taller tile saves a second of 128 rows: for gate/up 256 x 256
//     with one workgroup a CU, which also has room for the busiest expert's
//     rows, from 81 rows (105 rows each: 441 us, 128 x 128 472; 171 rows: 523 and
//     725; 209 rows: 563 and 779; 64 experts of 125 rows, K = 2048: 61.1 and
//     77.5); for a single product 192 x 128
//     (down of 64 experts, K = 1024, 125 rows each: 42.2 us, 256 x 256 43.8, 128 x
//     128 50.8; linear 300 x 49152 x 4096: 83 us, 128 x 128 104; 180 rows: 52 and 65;
//     6144 x 4096 x 4096, 1024 tiles: 107 and 120; 512 x 24576 x 6144, 576 tiles:
//     106 and 103).
//     As few tiles of 64 x 128 are still ahead of the kernel of few rows: 250 of
//     groups (24 experts, K = 832, 125 rows, 336 tiles: 11.6 us, 64 x 64 of that
//     kernel 16.5; 8 experts, K = 1024, 250 rows, 256 tiles: 11.1 and 12.7), 400 of a
//     linear layer (512 x 6144 x 6144, 384 tiles: 35.4 and 34.2; 768 rows: 45 and
//     52; 1000 x 2048 x 1024, 256 tiles: 9.7 and 8.6).
//   - A short K (a wave's share of it ends before its copies have got going)
//     and many tiles: its 64-row tiles with fewer rows too (down, K = 1792, 3 of 10
//     experts one row each: 46 us against 51).
//   - Else the largest tile of the few-rows kernel that still gives 300
//     workgroups: larger tiles copy the rows fewer times, but below about that
//     the chip's CUs are not all busy (linear 16 x 6144 x 6144: 32 channels
//     10.1 us, 64 11.6, 128 15.5; gate/up, 5 rows each: 373, 350, 349).
//   - Where no tile gives that many, eight waves on a long K keep twice as many
//     copies in flight on a CU (linear 1 x 6144 x 6144: 7.9 us, four waves 10.0;
//     K = 2048: 4.1 both; where the chip is full they lose: gate/up of 12
//     experts, one row each, 39.0 against 30.6).
template <bool DUAL, typename OUT>
hipError_t run_i8(const I8Params& p, int64_t rows, int64_t groups, int64_t mean, hipStream_t s) {
  const int64_t N = DUAL ? 2 * (int64_t)p.N : p.N;
  auto tiles = [&](int mt, int nt) { return groups * cdiv(mean, mt) * cdiv(N, nt); };
  if constexpr (DUAL) {
    if (mean > 80 && mean <= 224 && tiles(256, 256) >= 240)
      return run_mid<256, 256, 4, 2, 1, 3, DUAL, OUT>(p, rows, groups, mean, s);
  } else {
    if (p.offsets ? mean > 104 && mean <= 176 && tiles(192, 128) >= 400
                  : mean > 128 && tiles(192, 128) >= (mean <= 192 ? 360 : 700))
      return run_mid<192, 128, 2, 2, 2, 2, DUAL, OUT>(p, rows, groups, mean, s);
  }
  if (mean > 48 && tiles(128, 128) >= 400) return run_mid<128, 128, 2, 2, 2, 3, DUAL, OUT>(p, rows, groups, mean, s);
  const int64_t fill64 = p.offsets ? 250 : 400;
  if (mean > 32 ? tiles(64, 128) >= fill64 : p.K <= 2048 && tiles(64, 128) >= 1200)
    return run_mid<64, 128, 1, 4, 3, 2, DUAL, OUT>(p, rows, groups, mean, s);
  constexpr int64_t FILL = 300;
  if (mean > 32 && tiles(64, 64) >= FILL) return run_few<4, 4, 4, 2, DUAL, OUT>(p, rows, s);
  if (mean > 8) {
    if (mean <= 32 && tiles(32, 128) >= FILL) return run_few<2, 8, 4, 2, DUAL, OUT>(p, rows, s);
    if (tiles(32, 64) >= FILL) return run_few<2, 4, 4, 3, DUAL, OUT>(p, rows, s);
    if (tiles(32, 32) >= FILL) return run_few<2, 2, 4, 4, DUAL, OUT>(p, rows, s);
  } else {
    if (tiles(16, 128) >= FILL) return run_few<1, 8, 4, 2, DUAL, OUT>(p, rows, s);
    if (tiles(16, 64) >= FILL) return run_few<1, 4, 4, 3, DUAL, OUT>(p, rows, s);
  }
  if (p.K >= 4096) return run_few<1, 2, 8, 4, DUAL, OUT>(p, rows, s);
  return run_few<1, 2, 4, 4, DUAL, OUT>(p, rows, s);
}

// Whether a product goes to the tiles of gemm_dma.h (whole k-tiles of 128 codes,
// at least four) instead of the kernels above.  They run on one workgroup per CU,
// round by round, and for the experts they are ahead where there are some rounds
// of them (down of 8 experts, K = 8192, 500 rows each, 256 tiles: 191 us against
// 177; of 16, K = 2048, 512 tiles: 93 and 107) and groups have many rows (gate/up 206
// rows each 454 us against 439, 229 rows 624 and 612, 250 rows 704 and 761; down
// of K = 1536 206 rows 276 and 311); for down also where K is short and they are
// very many (K = 1792, 43 rows each 262 and 241, 63 rows 269 and 274, 105 rows 284
// and 324; gate/up, K = 2048, 83 rows, 1344 tiles: 207 and 162).
bool use_tiles(int64_t K, int64_t tiles, int64_t mean, bool dual) {
  if (K % 128 || K < 512) return false;
  return (mean > (dual ? 224 : 176) && tiles >= 400) || (!dual && K <= 2048 && mean > 56 && tiles >= 1024);
}

// The same for a linear layer: what decides is how much of the rounds its rows
// and channels fill, tiles that are not whole counted by what they have.  One
// round (K = 6144: 0.75 full 80 us against 90, 0.85 86 and 108; K = 2048, full: 47
// and 54; K = 4096, 256 rows, 0.75 65 and 75, 180 rows, 0.53 62 and 52, 128 rows 59
// and 40) or three (8192 x 4608 x 4096, 0.75: 160 and 177) from three quarters; two
// want more (K = 6144: 0.75 169 and 158, 0.92 168 and 189; K = 4096, 300 x 49152,
// 0.44: 116 and 83); a short K three full ones (8192 x 6144: K = 512 56 and 77, 1024
// 76 and 100).  One full round of a short K stays off them, although they are
// ahead there too (4096 x 4096: K = 512 31 and 33, 1024 37 and 42, 1536 43 and 52,
// 2048, where the limit is, 49 and 60).
// All without a bias.  With one the tiles are 10 to 57 % slower, the other kernel
// hardly at all, which the rule does not look at: 16384 x 6144 x 6144 bf16 665-677
// and 622-628, float32 633-644 and 643-650; 4096^3 97 and 96, 88 and 102; 8192 x
// 6144 x 2048 180 and 149, 155 and 156; 8192 x 4608 x 4096 245 and 189, 221 and 194.
bool use_tiles_linear(int64_t M, int64_t N, int64_t K) {
  if (K % 128 || K < 512) return false;
  const int64_t tiles = cdiv(M, 256) * cdiv(N, 256), rounds = cdiv(tiles, num_cus());
  const double full = (double)M * (double)N / ((double)rounds * num_cus() * 65536.0);
  return full >= (rounds == 2 ? 0.84 : 0.72) && (K >= 2048 || tiles >= 3 * num_cus());
}

// The local experts that have rows, as expected: a token's picks fall on num_local of E experts.
int64_t hit_experts(const moe_desc& d) {
  return std::min<int64_t>(d.num_local, std::max<int64_t>(1, (int64_t)d.T * d.k * d.num_local / d.E));
}

}  // namespace

hipError_t launch_i8_quantize_rows(const void* w, int dtype, int64_t rows, int64_t cols, int64_t ldw,
                                   const int32_t* nrows, int8_t* q, int64_t ldq, float* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == MOE_BF16)
    return quant_rows(reinterpret_cast<const uint16_t*>(w), rows, (int)cols, ldw, nrows, q, ldq, scale, s);
  return quant_rows(reinterpret_cast<const float*>(w), rows, (int)cols, ldw, nrows, q, ldq, scale, s);
}

hipError_t launch_gate_up_i8(const moe_desc& d, const int32_t* offsets, const int32_t* row_token, const int8_t* xq,
                             const float* xs, const int8_t* W1q, const float* W1s, const int8_t* W3q,
                             const float* W3s, void* gu, void* h, hipStream_t s) {
  I8Params p = {};
  p.x = xq;
  p.ldx = d.d;
  p.sx = xs;
  p.row_token = row_token;
  p.x_rows = d.T;
  p.w = W1q;
  p.w2 = W3q;
  p.ldw = d.d;
  p.sw = W1s;
  p.sw2 = W3s;
  p.offsets = offsets;
  p.ngroups = d.num_local;
  p.N = d.f;
  p.K = d.d;
  p.y = h;
  p.ldy = d.f;
  p.gu = reinterpret_cast<uint16_t*>(gu);
  const int64_t mean = cdiv((int64_t)d.T * d.k, d.E);
  if (use_tiles(d.d, d.num_local * cdiv(mean, 256) * cdiv(d.f, 128), mean, true))
    return launch_gate_up_i8_tiles(d, offsets, row_token, xq, xs, W1q, W1s, W3q, W3s, gu, h, s);
  return run_i8<true, uint16_t>(p, (int64_t)d.T * std::min(d.k, d.num_local), hit_experts(d), mean, s);
}

hipError_t launch_down_i8(const moe_desc& d, const int32_t* offsets, const int8_t* hq, const float* hs,
                          const int8_t* W2q, const float* W2s, void* y_perm, hipStream_t s) {
  I8Params p = {};
  p.x = hq;
  p.ldx = d.f;
  p.sx = hs;
  p.w = W2q;
  p.ldw = d.f;
  p.sw = W2s;
  p.offsets = offsets;
  p.ngroups = d.num_local;
  p.N = d.d;
  p.K = d.f;
  p.y = y_perm;
  p.ldy = d.d;
  const int64_t mean = cdiv((int64_t)d.T * d.k, d.E);
  if (use_tiles(d.f, d.num_local * cdiv(mean, 256) * cdiv(d.d, 256), mean, false))
    return launch_down_i8_tiles(d, offsets, hq, hs, W2q, W2s, y_perm, s);
  return run_i8<false, uint16_t>(p, (int64_t)d.T * std::min(d.k, d.num_local), hit_experts(d), mean, s);
}

hipError_t launch_i8_linear(int64_t M, int64_t N, int64_t K, const int8_t* xq, int64_t ldx, const float* xs,
                            const int8_t* wq, int64_t ldw, const float* ws, const float* bias, void* y, int64_t ldy,
                            int dtype, hipStream_t s) {
  if (M == 0) return hipSuccess;
  I8Params p = {};
  p.x = xq;
  p.ldx = ldx;
  p.sx = xs;
  p.w = wq;
  p.ldw = ldw;
  p.sw = ws;
  p.bias = bias;
  p.ngroups = 1;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.y = y;
  p.ldy = ldy;
  const int64_t esz = dtype == MOE_BF16 ? 2 : 4;
  // (the tiles store their output rows as 16-byte vectors)
  if (N * esz % 16 == 0 && ldy * esz % 16 == 0 && ldy <= 1 << 20 && use_tiles_linear(M, N, K))
    return launch_i8_linear_tiles((int)M, (int)N, (int)K, xq, ldx, xs, wq, ldw, ws, bias, y, ldy, dtype, s);
  if (dtype == MOE_BF16) return run_i8<false, uint16_t>(p, M, 1, M, s);
  return run_i8<false, float>(p, M, 1, M, s);
}

}  // namespace moe
