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
// every number).  code(v) is 127 v / max rounded to nearest, ties to even,
// exactly: r = v (127 / max) is off by at most 2^-23 of itself, so rint(r) is
// right unless r lies about that near to a tie (10^-6 of itself is asked).
// There, for float values, the quotient is taken in 64 bits, where none is
// nearer than 2^-40 of itself to a tie without being one.  For bf16 values, of
// 8 bits each, 254 v = (2n + 1) max is an equation of whole numbers up to
// 255^2 and a power of two, so none is nearer than 1.5 10^-5 of itself: what r
// cannot tell from a tie is one (v = max / 2 is: 63.5), and the even
// neighbour is 2 rint(r / 2).  A row of zeros has scale 0; a row with an
// infinity or a NaN has scale NaN and codes 0, so that what is computed from
// it is NaN.
struct RowQuant {
  float top, inv;
  bool small;  // 127 / max overflows: every quotient in 64 bits
  bool none;   // all codes are zero
  __device__ __forceinline__ explicit RowQuant(uint32_t bits) {
    top = __uint_as_float(bits);
    none = bits == 0 || bits >= 0x7f800000u;
    small = !none && top < 0x1p-100f;
    inv = none ? 0.f : 127.0f / top;
  }
  __device__ __forceinline__ float scale() const {
    return none && __float_as_uint(top) ? __uint_as_float(0x7fc00000u) : top / 127.0f;
  }
  template <bool EXACT>
  __device__ __forceinline__ int code(float v) const {
    const float r = v * inv;
    int q = (int)rintf(r);
    const bool tie = fabsf(fabsf(r - truncf(r)) - 0.5f) < 1e-6f * fabsf(r);
    if (!EXACT && tie) q = 2 * (int)rintf(r * 0.5f);
    if (EXACT && tie) q = (int)rint((double)v * 127.0 / (double)top);
    if (small) q = (int)rint((double)v * 127.0 / (double)top);
    return none ? 0 : q;
  }
};

// One wave per row.  NV > 0: the row is held in NV vectors per lane and read
// once; NV = 0: any length, read twice (the second time from cache).  VEC:
// rows start at multiples of 16 bytes, so the values come as vectors (the last
// may reach past the row's end, never past the 16 aligned bytes that hold its
// last value).  nrows (device, or NULL): rows at or past it are left alone.
// Bound by HBM: (b + 1) bytes a value.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(256) i8_quant_rows_kernel(const T* __restrict__ w, int64_t rows, int64_t cols,
                                                            int64_t ldw, const int32_t* __restrict__ nrows,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
  constexpr int N = 16 / sizeof(T);
  constexpr bool EXACT = sizeof(T) == 4;
  const int lane = threadIdx.x & 63;
  const int64_t lim = nrows ? min(rows, (int64_t)max(*nrows, 0)) : rows;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < lim; r += (int64_t)gridDim.x * 4) {
    const T* src = w + r * ldw;
    int8_t* dst = q + r * ldq;
    if constexpr (VEC) {
      u32x4_t held[NV > 0 ? NV : 1];
      uint32_t top = 0;
      auto load = [&](int64_t c) -> u32x4_t {  // columns c .. c + N - 1, zero past the end
        u32x4_t x = {0, 0, 0, 0};
        if (c < cols) x = *reinterpret_cast<const u32x4_t*>(src + c);
        if (c + N > cols) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (sizeof(T) == 4) {
              if (c + i >= cols) x[i] = 0;
            } else {
              if (c + 2 * i >= cols) x[i] = 0;
              else if (c + 2 * i + 1 >= cols) x[i] &= 0xffffu;
            }
          }
        }
        return x;
      };
      auto grow = [&](u32x4_t x) {
        float v[N];
        unpack(x, v);
#pragma unroll
        for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) held[j] = load((int64_t)(j * 64 + lane) * N);
#pragma unroll
        for (int j = 0; j < NV; ++j) grow(held[j]);
      } else {
        for (int64_t c = (int64_t)lane * N; c < cols; c += 64 * N) grow(load(c));
      }
      const RowQuant rq(wave_max(top));
      auto put = [&](int64_t c, u32x4_t x) {
        if (c >= cols) return;
        float v[N];
        unpack(x, v);
        uint32_t o[N / 4];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t b = (uint32_t)rq.template code<EXACT>(v[i]) & 0xffu;
          o[i / 4] = i % 4 ? o[i / 4] | (b << (8 * (i % 4))) : b;
        }
        if (c + N <= cols) {
          if constexpr (N == 8) *reinterpret_cast<u32x2_t*>(dst + c) = u32x2_t{o[0], o[1]};
          else *reinterpret_cast<uint32_t*>(dst + c) = o[0];
        } else {
          for (int i = 0; c + i < cols; ++i) dst[c + i] = (int8_t)(o[i / 4] >> (8 * (i % 4)));
        }
      };
      if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) put((int64_t)(j * 64 + lane) * N, held[j]);
      } else {
        for (int64_t c = (int64_t)lane * N; c < cols; c += 64 * N) put(c, load(c));
      }
      if (lane == 0) scale[r] = rq.scale();
    } else {
      uint32_t top = 0;
      for (int64_t c = lane; c < cols; c += 64)
        top = max(top, __float_as_uint(Elem<T>::ld(src, c)) & 0x7fffffffu);
      const RowQuant rq(wave_max(top));
      for (int64_t c = lane; c < cols; c += 64) dst[c] = (int8_t)rq.template code<EXACT>(Elem<T>::ld(src, c));
      if (lane == 0) scale[r] = rq.scale();
    }
  }
}

template <typename T>
hipError_t quant_rows(const T* w, int64_t rows, int64_t cols, int64_t ldw, const int32_t* nrows, int8_t* q,
                      int64_t ldq, float* scale, hipStream_t s) {
  constexpr int64_t N = 16 / sizeof(T);
  const int64_t nv = (cols + 64 * N - 1) / (64 * N);  // vectors per lane
  const unsigned grid = (unsigned)std::min<int64_t>((rows + 3) / 4, (int64_t)num_cus() * 16);
#define MOE_I8_QUANT(NV, VEC) \
  i8_quant_rows_kernel<T, NV, VEC><<<grid, 256, 0, s>>>(w, rows, cols, ldw, nrows, q, ldq, scale)
  if (ldw % N) MOE_I8_QUANT(0, false);
  else if (nv <= 4) MOE_I8_QUANT(4, true);
  else if (nv <= 12) MOE_I8_QUANT(12, true);
  else MOE_I8_QUANT(0, true);
#undef MOE_I8_QUANT
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
  int64_t tiles;  // m-tile slots times channel tiles
  void* y;
  int64_t ldy;
  uint16_t* gu;
};

// With few rows the product streams the weights, each of whose bytes is used
// by one workgroup only: the kernel is bound by HBM and has to keep many loads
// in flight.  A workgroup computes MB*16 rows x NB*16 channels (DUAL: half of
// them gate, half up) over all of K, cut into chunks of 128 codes that its
// four waves take in turn; no wave shares an operand with another, so the main
// loop has no barrier: each wave copies its own chunks into its own LDS ring
// (LDS DMA, 8 rows x 128 bytes per instruction, all lines whole) and waits for
// its own copies only.  The four partial sums are whole numbers and are added
// through LDS at the end, in any order with the same result.
//   Fragments: v_mfma_i32_16x16x64_i8 with the channels as rows and the tokens
//   as columns; lane l holds 16 codes of row l % 16 at k = 16 (l / 16), and
//   the result's rows 4 (l / 16) .. + 3 of column l % 16, so a lane's four
//   sums are consecutive channels of one token.
//   LDS: rows of 128 bytes, 16-byte piece c of row r at c ^ swz_k(r).
template <int MB, int NB, int NST, bool DUAL, typename OUT>
__global__ void __launch_bounds__(256) i8_few_rows_kernel(I8Params p) {
  using namespace dma;
  static_assert(!DUAL || NB % 2 == 0, "gate and up blocks");
  constexpr int MT = MB * 16, NT = NB * 16;
  constexpr int OC = DUAL ? NT / 2 : NT;       // output channels
  constexpr int STAGE = (MT + NT) * 128;       // bytes: weight rows, then token rows
  constexpr int PER = (MT + NT) / 8;           // copies per chunk
  constexpr int RP = NT + 4;                   // pitch of the partial sums (ints)
  constexpr int RING = 4 * NST * STAGE, RED = 4 * MT * RP * 4;
  static_assert(PER * (NST - 1) < 64, "vmcnt range");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > RED ? RING : RED];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ntiles = (p.N + OC - 1) / OC;
  for (int64_t id = blockIdx.x; id < p.tiles; id += gridDim.x) {
    const int ntile = (int)(id % ntiles);
    const int slot = (int)(id / ntiles);

    // The slot's group and m-tile: groups have ceil(rows / MT) m-tiles each, in
    // order.  Every wave searches alike, 64 groups at a time.
    int g = 0, m0 = slot * MT, m1 = p.M;
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
          const int mt = slot - before - (__shfl(inc, l, WAVE) - __shfl(c, l, WAVE));
          m0 = __shfl(lo, l, WAVE) + mt * MT;
          m1 = __shfl(hi, l, WAVE);
          break;
        }
        before += __shfl(inc, 63, WAVE);
      }
      if (g < 0) break;  // more slots than m-tiles (and every later slot is past them too)
    }
    g = __builtin_amdgcn_readfirstlane(g);
    m0 = __builtin_amdgcn_readfirstlane(m0);
    const int mlim = __builtin_amdgcn_readfirstlane(min(MT, m1 - m0));
    const int n0 = ntile * OC, nlim = min(OC, p.N - n0);

    // Copy offsets.  Copy j moves LDS rows 8j .. 8j + 7: lane i row 8j + i/8,
    // position i % 8, which holds piece (i % 8) ^ swz_k(row) of the row's 128
    // bytes.  Rows that do not exist get bit 31, past every resource: zeros.
    const i32x4 rw = make_rsrc(p.w + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw);
    const i32x4 rw2 = DUAL ? make_rsrc(p.w2 + ((int64_t)g * p.N + n0) * p.ldw, (uint64_t)nlim * p.ldw) : rw;
    const i32x4 rx = p.row_token ? make_rsrc(p.x, (uint64_t)p.x_rows * p.ldx)
                                 : make_rsrc(p.x + (int64_t)m0 * p.ldx, (uint64_t)mlim * p.ldx);
    uint32_t vw[NT / 8], vx[MT / 8];
    auto piece = [&](int row) { return (lane & 7) ^ swz_k<64>(row); };
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
    const int mine = (chunks - wave + 3) / 4;  // chunks wave, wave + 4, ...
    const uint32_t ring = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem) + wave * NST * STAGE;
    auto copy = [&](int i) {  // the wave's chunk i into stage i % NST
      const int k0 = (wave + 4 * i) * 128;
      const uint32_t st = ring + (i % NST) * STAGE;
      const bool whole = k0 + 128 <= p.K;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const bool tok = j >= NT / 8;
        uint32_t v = tok ? vx[tok ? j - NT / 8 : 0] : vw[tok ? 0 : j];
        // (a piece past K lies in the next row: none of it is wanted)
        if (!whole && k0 + piece(8 * (tok ? j - NT / 8 : j) + (lane >> 3)) * 16 >= p.K) v = 0x80000000u;
        const i32x4 r = tok ? rx : (DUAL && j >= NT / 16 ? rw2 : rw);
        dma16(r, v, (uint32_t)k0, __builtin_amdgcn_readfirstlane(st + j * 1024));
      }
    };

    i32x4_t acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int b = 0; b < MB; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};

#pragma unroll
    for (int i = 0; i < NST; ++i)
      if (i < mine) copy(i);
    for (int i = 0; i < mine; ++i) {
      wait_stages<PER, NST - 1>(min(NST - 1, mine - 1 - i));
      asm volatile("" ::: "memory");
      const uint8_t* st = smem + (wave * NST + i % NST) * STAGE;
      i32x4_t fw[2][NB], fx[2][MB];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int r = b * 16 + (lane & 15);
          fx[ks][b] = *reinterpret_cast<const i32x4_t*>(st + NT * 128 + r * 128 +
                                                        (((4 * ks + (lane >> 4)) ^ swz_k<64>(r)) << 4));
        }
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const int r = a * 16 + (lane & 15);
          fw[ks][a] =
              *reinterpret_cast<const i32x4_t*>(st + r * 128 + (((4 * ks + (lane >> 4)) ^ swz_k<64>(r)) << 4));
        }
      }
      // The stage is read before its next copy is issued.
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      asm volatile("" ::: "memory");
      if (i + NST < mine) copy(i + NST);
      if ((wave + 4 * i) * 128 + 128 > p.K && p.K % 16) {
        // the codes past K in the row's last piece are not the caller's to give:
        // zeroed in one operand, the other's do not matter
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const int left = p.K - ((wave + 4 * i) * 128 + ks * 64 + (lane >> 4) * 16);  // valid codes of the lane's 16
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int v = left - 4 * d;
            const uint32_t keep = v >= 4 ? 0xffffffffu : v <= 0 ? 0u : (1u << (8 * v)) - 1u;
#pragma unroll
            for (int b = 0; b < MB; ++b) fx[ks][b][d] &= (int)keep;
          }
        }
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int a = 0; a < NB; ++a)
#pragma unroll
          for (int b = 0; b < MB; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[ks][a], fx[ks][b], acc[a][b], 0, 0, 0);
    }

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
      for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const i32x4_t*>(red + (w * MT + row) * RP + c);
      return v;
    };
    constexpr int VPR = OC / 4;  // vectors of four channels per row
    const bool vec = p.N % 4 == 0 && p.ldy % 4 == 0;  // (then a vector is whole or outside, and aligned)
    for (int e = tid; e < mlim * VPR; e += 256) {
      const int row = e / VPR, c = (e % VPR) * 4;
      if (c >= nlim) continue;
      const int64_t r = (int64_t)m0 + row;
      const float sx = p.sx[p.row_token ? p.row_token[r] : r];
      const i32x4_t s1 = total(row, c);
      float o[4];
      const int64_t ch = (int64_t)g * p.N + n0 + c;
      if constexpr (DUAL) {
        const i32x4_t s2 = total(row, OC + c);
        float gt[4], up[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // (N is a multiple of 64)
          gt[q] = (float)s1[q] * sx * p.sw[ch + q];
          up[q] = (float)s2[q] * sx * p.sw2[ch + q];
          o[q] = gt[q] * sigmoidf_(gt[q]) * up[q];
        }
        if (p.gu) {
          uint16_t* gr = p.gu + r * 2 * p.N + n0 + c;
          *reinterpret_cast<u32x2_t*>(gr) = u32x2_t{pack_bf2(gt[0], gt[1]), pack_bf2(gt[2], gt[3])};
          *reinterpret_cast<u32x2_t*>(gr + p.N) = u32x2_t{pack_bf2(up[0], up[1]), pack_bf2(up[2], up[3])};
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (c + q >= nlim) break;
          o[q] = (float)s1[q] * sx * p.sw[ch + q];
          if (p.bias) o[q] += p.bias[ch + q];
        }
      }
      OUT* y = reinterpret_cast<OUT*>(p.y) + r * p.ldy + n0 + c;
      if (vec) {
        if constexpr (sizeof(OUT) == 2)
          *reinterpret_cast<u32x2_t*>(y) = u32x2_t{pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3])};
        else *reinterpret_cast<f32x4_t*>(y) = f32x4_t{o[0], o[1], o[2], o[3]};
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < nlim) Elem<OUT>::st(y, q, o[q]);
      }
    }
    __syncthreads();  // the next tile's copies overwrite the partial sums
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int MB, int NB, int NST, bool DUAL, typename OUT>
hipError_t run_few(I8Params p, int64_t rows, hipStream_t s) {
  constexpr int OC = NB * 16 / (DUAL ? 2 : 1);
  // m-tiles at most: every group may end in a partial one
  const int64_t slots = p.offsets ? rows / (MB * 16) + std::min<int64_t>(p.ngroups, rows) : cdiv(rows, MB * 16);
  p.tiles = slots * cdiv(p.N, OC);
  const unsigned grid = (unsigned)std::min<int64_t>(p.tiles, 1 << 22);  // (a launch has fewer than 2^32 threads)
  i8_few_rows_kernel<MB, NB, NST, DUAL, OUT><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

// rows: an upper bound of all rows; mean: the expected rows of a group.
template <bool DUAL, typename OUT>
hipError_t run_i8(const I8Params& p, int64_t rows, int64_t mean, hipStream_t s) {
  if (mean <= 16) return run_few<1, 4, 2, DUAL, OUT>(p, rows, s);
  return run_few<4, 4, 2, DUAL, OUT>(p, rows, s);
}

}  // namespace

hipError_t launch_i8_quantize_rows(const void* w, int dtype, int64_t rows, int64_t cols, int64_t ldw,
                                   const int32_t* nrows, int8_t* q, int64_t ldq, float* scale, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == MOE_BF16)
    return quant_rows(reinterpret_cast<const uint16_t*>(w), rows, cols, ldw, nrows, q, ldq, scale, s);
  return quant_rows(reinterpret_cast<const float*>(w), rows, cols, ldw, nrows, q, ldq, scale, s);
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
  if (d.d % 128 == 0 && d.d >= 512 && mean > 64)
    return launch_gate_up_i8_tiles(d, offsets, row_token, xq, xs, W1q, W1s, W3q, W3s, gu, h, s);
  return run_i8<true, uint16_t>(p, (int64_t)d.T * std::min(d.k, d.num_local), mean, s);
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
  if (d.f % 128 == 0 && d.f >= 512 && mean > 64)
    return launch_down_i8_tiles(d, offsets, hq, hs, W2q, W2s, y_perm, s);
  return run_i8<false, uint16_t>(p, (int64_t)d.T * std::min(d.k, d.num_local), mean, s);
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
  if (K % 128 == 0 && K >= 512 && N * esz % 16 == 0 && ldy * esz % 16 == 0 && ldy <= 1 << 20 &&
      cdiv(M, 256) * cdiv(N, 256) >= 128)
    return launch_i8_linear_tiles((int)M, (int)N, (int)K, xq, ldx, xs, wq, ldw, ws, bias, y, ldy, dtype, s);
  if (dtype == MOE_BF16) return run_i8<false, uint16_t>(p, M, M, s);
  return run_i8<false, float>(p, M, M, s);
}

}  // namespace moe
