// Weights in 4 bits with a scale per group of a row: the quantiser, its
// inverse and the linear layer.
//
// A group's values v are held as codes q and one float32 scale s = max|v| / 7,
// q = 7 v / max|v| rounded to nearest, ties to even; v is about s q.  Eight
// codes share a 32-bit word, code i (plus 8) at bit 4 (i / 2 + 4 (i % 2)):
// the word's pairs of neighbours then lie 16 bits apart, as two bf16 values of
// a register do.
#include <algorithm>

#include "internal.h"
#include "stream.h"

namespace moe {

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Position of a row's word: thread i of the grid has word i % wpr of row i / wpr,
// where wpr counts whole groups (a group's lanes lie together).  The row of the
// workgroup's first thread in 64 bits once, then 32.
__device__ __forceinline__ void word_of(int64_t tile, uint32_t wpr, int64_t& row, uint32_t& word) {
  const uint64_t first = (uint64_t)tile * 256;
  const uint64_t r0 = first / wpr;
  const uint32_t w = (uint32_t)(first - r0 * wpr) + threadIdx.x;
  row = (int64_t)r0 + w / wpr;
  word = w % wpr;
}

// A group's codes from its largest |value| m: r = v (7 / m) is off by less than
// 2 10^-6, so the integer nearest to r is right unless r lies within 10^-5 of a
// tie.  There, for float values, the quotient is taken in 64 bits, where none
// is nearer than 2^-29 of itself to a tie without being one.  For bf16 values,
// of 8 bits each, 14 v = (2n + 1) m is an equation of whole numbers up to 7140
// and a power of two, so no quotient lies within 6 10^-5 of a tie without being
// one, and the even neighbour is 2 rint(r / 2).
template <bool EXACT>
__device__ __forceinline__ uint32_t i4_codes(const float (&v)[8], uint32_t bits) {
  const float top = __uint_as_float(bits);
  if (bits == 0 || bits >= 0x7f800000u) return 0x88888888u;
  const bool small = top < 0x1p-100f;  // (7 / m may overflow: every quotient in 64 bits)
  const float inv = small ? 0.f : 7.0f / top;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = v[i] * inv;
    float q = rintf(r);
    if (small) {
      q = (float)rint((double)v[i] * 7.0 / (double)top);
    } else if (fabsf(r - q) > 0.49999f) {
      if (EXACT) q = (float)rint((double)v[i] * 7.0 / (double)top);
      else q = 2.f * rintf(0.5f * r);
    }
    word |= (uint32_t)((int)q + 8) << (4 * ((i >> 1) + 4 * (i & 1)));
  }
  return word;
}

// One word of codes per thread, a group's words on neighbouring lanes.  Bound
// by HBM: b + 1/2 + 4/g bytes a value.  VEC: rows start at multiples of 16
// bytes.
template <typename T, int GRP, bool VEC>
__global__ void __launch_bounds__(256) i4_quantize_kernel(const T* __restrict__ w, int64_t rows, uint32_t words,
                                                          uint32_t wpr, int64_t ldw, uint8_t* __restrict__ q,
                                                          int64_t ldq, float* __restrict__ scale, int64_t lds,
                                                          int64_t tiles) {
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int64_t row;
    uint32_t word;
    word_of(tile, wpr, row, word);
    const bool in = row < rows && word < words;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (in) {
      const T* src = w + row * ldw + (int64_t)word * 8;
      if constexpr (VEC && sizeof(T) == 2) {
        Vec16<uint16_t>::load(src, v);
      } else if constexpr (VEC) {
        float a[4], b[4];
        Vec16<float>::load(src, a);
        Vec16<float>::load(src + 4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Elem<T>::ld(src, i);
      }
    }
    uint32_t top = 0;  // as bits, so that NaN > infinity > every number
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = GRP / 16; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, WAVE));
    if (in) {
      *reinterpret_cast<uint32_t*>(q + row * ldq + (int64_t)word * 4) = i4_codes<sizeof(T) == 4>(v, top);
      if (word % (GRP / 8) == 0)
        scale[row * lds + word / (GRP / 8)] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                                 : __uint_as_float(top) / 7.0f;
    }
  }
}

// One word of codes per thread -> eight values.  Bound by HBM.
template <typename T, int GRP, bool VEC>
__global__ void __launch_bounds__(256) i4_dequantize_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                            const float* __restrict__ scale, int64_t lds, int64_t rows,
                                                            uint32_t words, T* __restrict__ w, int64_t ldw,
                                                            int64_t tiles) {
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int64_t row;
    uint32_t word;
    word_of(tile, words, row, word);
    if (row >= rows) continue;
    const uint32_t c = *reinterpret_cast<const uint32_t*>(q + row * ldq + (int64_t)word * 4);
    const float s = scale[row * lds + word / (GRP / 8)];
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s * (float)((int)((c >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15u) - 8);
    T* dst = w + row * ldw + (int64_t)word * 8;
    if constexpr (VEC && sizeof(T) == 2) {
      Vec16<uint16_t>::store(dst, v);
    } else if constexpr (VEC) {
      *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) Elem<T>::st(dst, i, v[i]);
    }
  }
}

unsigned grid_of(int64_t tiles) { return (unsigned)std::min<int64_t>(tiles, (int64_t)num_cus() * 64); }

template <typename T, int GRP>
hipError_t quantize(const T* w, int64_t rows, int64_t cols, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                    int64_t lds, hipStream_t s) {
  const uint32_t words = (uint32_t)(cols / 8), wpr = (uint32_t)(cdiv(cols, GRP) * (GRP / 8));
  const int64_t tiles = cdiv(rows * wpr, 256);
  if (ldw % (int64_t)(16 / sizeof(T)) == 0)
    i4_quantize_kernel<T, GRP, true><<<grid_of(tiles), 256, 0, s>>>(w, rows, words, wpr, ldw, q, ldq, scale, lds, tiles);
  else
    i4_quantize_kernel<T, GRP, false><<<grid_of(tiles), 256, 0, s>>>(w, rows, words, wpr, ldw, q, ldq, scale, lds, tiles);
  return hipGetLastError();
}

template <typename T, int GRP>
hipError_t dequantize(const uint8_t* q, int64_t ldq, const float* scale, int64_t lds, int64_t rows, int64_t cols, T* w,
                      int64_t ldw, hipStream_t s) {
  const uint32_t words = (uint32_t)(cols / 8);
  const int64_t tiles = cdiv(rows * words, 256);
  if (ldw % (int64_t)(16 / sizeof(T)) == 0)
    i4_dequantize_kernel<T, GRP, true><<<grid_of(tiles), 256, 0, s>>>(q, ldq, scale, lds, rows, words, w, ldw, tiles);
  else
    i4_dequantize_kernel<T, GRP, false><<<grid_of(tiles), 256, 0, s>>>(q, ldq, scale, lds, rows, words, w, ldw, tiles);
  return hipGetLastError();
}

// The linear layer: a workgroup computes RB rows x R channels over all of K, whose
// stretches of 256 its W waves take in turn, each through a ring of S stages
// (stream.h).
struct LinearParams {
  const uint16_t* x;
  const uint8_t* w;
  const float* s;
  const float* bias;
  void* y;
  int64_t ldx, ldw, lds, ldy;
  int M, N, K;
  int mblocks, ntiles;
  int64_t items;
};

template <int GRP, int RB, int R, int W, int S, typename OUT>
__global__ void __launch_bounds__(64 * W) i4_linear_kernel(LinearParams p) {
  using namespace stream;
  using ST = Stage<GRP, R, 1, false, RB>;
  constexpr int RED = W * RB * (R + 4) * 4;
  constexpr int RING = W * S * ST::BYTES;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > RED ? RING : RED];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Blocks of rows that share channels run side by side on one XCD (workgroups
  // go to the eight in turn), whose L2 serves the weights to all but the first.
  for (int64_t id = blockIdx.x; id < p.items; id += gridDim.x) {
  const int mb = (int)((id >> 3) % p.mblocks);
  const int64_t tile = (id >> 3) / p.mblocks * 8 + (id & 7);
  if (tile >= p.ntiles) continue;
  const int m0 = mb * RB, rows = min(RB, p.M - m0), n0 = (int)tile * R, chans = min(R, p.N - n0);

  Source src;
  src.w[0] = src.w[1] = make_rsrc(p.w + n0 * p.ldw, (uint64_t)(chans - 1) * p.ldw + p.K / 2);
  src.s[0] = src.s[1] = make_rsrc(p.s + n0 * p.lds, (uint64_t)chans * p.lds * 4);
  src.x = make_rsrc(p.x + m0 * p.ldx, (uint64_t)rows * p.ldx * 2);
  src.pitch = (uint32_t)p.ldw;
  src.spitch = (uint32_t)p.lds * 4;
  src.K = p.K;
  src.rows = chans;
  uint32_t xr[ST::XI];
#pragma unroll
  for (int n = 0; n < ST::XI; ++n) {
    xr[n] = (uint32_t)(ST::x_row(n, lane) * p.ldx * 2);
  }
  const uint32_t ring = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem) + wave * S * ST::BYTES;
  const uint8_t* ring_p = smem + wave * S * ST::BYTES;
  const int chunks = (p.K + 255) / 256;
  const int mine = (chunks - wave + W - 1) / W;  // stretches wave, wave + W, ...
  auto copy = [&](int i, int slot) {
    const int k0 = __builtin_amdgcn_readfirstlane((wave + W * i) * 256);
    const uint32_t at = __builtin_amdgcn_readfirstlane(ring + slot * ST::BYTES);
    ST::copy_w(src, k0, at, lane);
    ST::copy_x(src, xr, rows, k0, at, lane);
  };
  const int per = ST::WI + ST::SI + (rows * ST::XROW + 1023) / 1024;  // copies of a stage
  f32x4_t acc[ST::RT];
#pragma unroll
  for (int t = 0; t < ST::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (i < mine) copy(i, i);
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    wait_younger<(S - 1) * (ST::WI + ST::SI + ST::XI)>((min(i + S, mine) - i - 1) * per);
    ST st;
    st.read(ring_p + slot * ST::BYTES, lane);
    if (!ST::EARLY) st.multiply(acc, lane);
    reads_done();
    if (i + S < mine) copy(i + S, slot);
    if (ST::EARLY) st.multiply(acc, lane);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  // Partial sums [wave][row][channel] over the ring, once every wave is done with it.
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  const int col = lane & 15;
  if (col < RB && (R > 8 || lane < 32)) {
#pragma unroll
    for (int t = 0; t < ST::RT; ++t)
      *reinterpret_cast<f32x4_t*>(red + (wave * RB + col) * (R + 4) + 16 * t + 4 * (lane >> 4)) = acc[t];
  }
  __syncthreads();
  for (int i = tid; i < rows * R; i += 64 * W) {
    const int row = i / R, c = i % R;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[(w * RB + row) * (R + 4) + c];
    if (c < chans) Elem<OUT>::st((OUT*)p.y + (m0 + row) * p.ldy, n0 + c, p.bias ? sum + p.bias[n0 + c] : sum);
  }
  __syncthreads();  // the next tile's copies overwrite the partial sums
  }
}

template <int GRP, int RB, int R, int W, int S, typename OUT>
hipError_t run_linear(LinearParams p, hipStream_t s) {
  p.mblocks = (int)cdiv(p.M, RB);
  p.ntiles = (int)cdiv(p.N, R);
  p.items = cdiv(p.ntiles, 8) * 8 * p.mblocks;
  const unsigned grid = (unsigned)std::min<int64_t>(p.items, 1 << 22);
  i4_linear_kernel<GRP, RB, R, W, S, OUT><<<grid, 64 * W, 0, s>>>(p);
  return hipGetLastError();
}

template <int GRP, typename OUT>
hipError_t linear(const LinearParams& p, hipStream_t s) {
  if (p.M == 1) return run_linear<GRP, 1, 16, 8, 2, OUT>(p, s);
  if (p.M <= 4) return run_linear<GRP, 4, 16, 8, 2, OUT>(p, s);
  if (p.M <= 16) return run_linear<GRP, 16, 32, 4, 2, OUT>(p, s);
  return run_linear<GRP, 16, 64, 4, 2, OUT>(p, s);
}

}  // namespace

hipError_t launch_i4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t ldw, int group, uint8_t* q,
                              int64_t ldq, float* scale, int64_t lds, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  auto run = [&](auto* p) {
    return group == 32   ? quantize<std::remove_pointer_t<decltype(p)>, 32>(p, rows, cols, ldw, q, ldq, scale, lds, s)
           : group == 64 ? quantize<std::remove_pointer_t<decltype(p)>, 64>(p, rows, cols, ldw, q, ldq, scale, lds, s)
                         : quantize<std::remove_pointer_t<decltype(p)>, 128>(p, rows, cols, ldw, q, ldq, scale, lds, s);
  };
  return dtype == MOE_F32 ? run(const_cast<float*>((const float*)w)) : run(const_cast<uint16_t*>((const uint16_t*)w));
}

hipError_t launch_i4_dequantize(const uint8_t* q, int64_t ldq, const float* scale, int64_t lds, int64_t rows,
                                int64_t cols, int group, void* w, int dtype, int64_t ldw, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  auto run = [&](auto* p) {
    return group == 32   ? dequantize<std::remove_pointer_t<decltype(p)>, 32>(q, ldq, scale, lds, rows, cols, p, ldw, s)
           : group == 64 ? dequantize<std::remove_pointer_t<decltype(p)>, 64>(q, ldq, scale, lds, rows, cols, p, ldw, s)
                         : dequantize<std::remove_pointer_t<decltype(p)>, 128>(q, ldq, scale, lds, rows, cols, p, ldw, s);
  };
  return dtype == MOE_F32 ? run((float*)w) : run((uint16_t*)w);
}

hipError_t launch_i4_linear(int64_t M, int64_t N, int64_t K, int group, const void* x, int64_t ldx, const uint8_t* wq,
                            int64_t ldw, const float* ws, int64_t lds, const float* bias, void* y, int64_t ldy,
                            int dtype, hipStream_t s) {
  if (M == 0) return hipSuccess;
  const LinearParams p{(const uint16_t*)x, wq, ws, bias, y, ldx, ldw, lds, ldy, (int)M, (int)N, (int)K, 0, 0, 0};
  auto run = [&](auto o) {
    using OUT = decltype(o);
    return group == 32 ? linear<32, OUT>(p, s) : group == 64 ? linear<64, OUT>(p, s) : linear<128, OUT>(p, s);
  };
  return dtype == MOE_F32 ? run(0.f) : run((uint16_t)0);
}

}  // namespace moe
