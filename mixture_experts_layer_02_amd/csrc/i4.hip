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

// A thread's place among the pieces of all rows: piece i of the grid's threads is
// piece i % per of row i / per; the next one lies `step` threads on, reached with
// adds (a division each time cost as much as the rest).
struct Place {
  int64_t row, rows;
  uint32_t at, per, d_at;
  int64_t d_row;
  __device__ __forceinline__ Place(int64_t rows_, uint32_t per_) : rows(rows_), per(per_) {
    const uint64_t first = (uint64_t)blockIdx.x * 256, r0 = first / per, step = (uint64_t)gridDim.x * 256;
    const uint32_t w = (uint32_t)(first - r0 * per) + threadIdx.x;
    row = (int64_t)r0 + w / per;
    at = w % per;
    d_row = (int64_t)(step / per);
    d_at = (uint32_t)(step - (uint64_t)d_row * per);
  }
  __device__ __forceinline__ void next() {
    row += d_row, at += d_at;
    if (at >= per) at -= per, ++row;
  }
};

// A group's codes from its largest |value| m: r = v (7 / m) is off by less than
// 2 10^-6, so the integer nearest to r is right unless r lies within 10^-5 of a
// tie.  There, for float values, the quotient is taken in 64 bits, where none
// is nearer than 2^-29 of itself to a tie without being one.  For bf16 values,
// of 8 bits each, 14 v = (2n + 1) m is an equation of whole numbers up to 7140
// and a power of two, so no quotient lies within 6 10^-5 of a tie without being
// one, and the even neighbour is 2 rint(r / 2).  r + 1.5 2^23 + 8 rounds r to
// the nearest integer, ties to even, in the low bits of its own bit pattern.
template <bool EXACT>
__device__ __forceinline__ uint32_t i4_codes(const float (&v)[8], uint32_t bits) {
  constexpr float MAGIC = 12582912.0f + 8.0f;
  const float top = __uint_as_float(bits);
  const bool none = bits == 0 || bits >= 0x7f800000u;
  const bool small = top < 0x1p-100f;  // (7 / m may overflow: every quotient in 64 bits)
  const float inv = none || small ? 0.f : 7.0f / top;
  uint32_t b[8];
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = none ? 0.f : v[i] * inv, m = r + MAGIC;
    b[i] = __float_as_uint(m);
    off = fmaxf(off, fabsf(r - (m - MAGIC)));
  }
  if (!none && (off > 0.49999f || small)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = v[i] * inv;
      float q = rintf(r);
      if (small) q = (float)rint((double)v[i] * 7.0 / (double)top);
      else if (fabsf(r - q) > 0.49999f) q = EXACT ? (float)rint((double)v[i] * 7.0 / (double)top) : 2.f * rintf(0.5f * r);
      b[i] = (uint32_t)((int)q + 8);
    }
  }
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= (b[i] & 15u) << (4 * ((i >> 1) + 4 * (i & 1)));
  return word;
}

constexpr int UNROLL = 2;  // words of a thread that are read before the first is used

// One word of codes per thread, a group's words on neighbouring lanes.  Bound
// by HBM, b + 1/2 + 4/g bytes a value (196608 x 1792 bf16: 222 us, 4.1 TB/s, where a
// copy runs at 5.1; a workgroup for every 512 words, none twice: 242 us).  VEC: rows start at multiples of 16
// bytes.
template <typename T, int GRP, bool VEC>
__global__ void __launch_bounds__(256) i4_quantize_kernel(const T* __restrict__ w, int64_t rows, uint32_t words,
                                                          uint32_t wpr, int64_t ldw, uint8_t* __restrict__ q,
                                                          int64_t ldq, float* __restrict__ scale, int64_t lds,
                                                          int64_t turns) {
  Place at(rows, wpr);  // (wpr counts whole groups: a group's lanes lie together)
  for (int64_t turn = 0; turn < turns; ++turn) {
    float v[UNROLL][8];
    int64_t row[UNROLL];
    uint32_t word[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      row[u] = at.row, word[u] = at.at;
      at.next();
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      if (row[u] < rows && word[u] < words) {
        const T* src = w + row[u] * ldw + (int64_t)word[u] * 8;
        if constexpr (VEC && sizeof(T) == 2) {
          const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][2 * i] = __uint_as_float(a[i] << 16), v[u][2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        } else if constexpr (VEC) {
          const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src));
          const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src + 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = a[i], v[u][4 + i] = b[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] = Elem<T>::ld(src, i);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      uint32_t top = 0;  // as bits, so that NaN > infinity > every number
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[u][i]) & 0x7fffffffu);
#pragma unroll
      for (int o = GRP / 16; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, WAVE));
      const uint32_t code = i4_codes<sizeof(T) == 4>(v[u], top);
      if (row[u] < rows && word[u] < words) {
        *reinterpret_cast<uint32_t*>(q + row[u] * ldq + (int64_t)word[u] * 4) = code;
        if (word[u] % (GRP / 8) == 0)
          scale[row[u] * lds + word[u] / (GRP / 8)] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                                                         : __uint_as_float(top) / 7.0f;
      }
    }
  }
}

// 16 bytes of values per thread: a word's eight in bf16, half a word's four in
// float32.  Bound by HBM (196608 x 1792 to float32: 357 us, 4.5 TB/s, to bf16 194;
// with stores that stay in the L2 382 and 198, 1792 x 6144 to float32 15.4 in place of
// 9.4; with as few workgroups as the quantiser 418 and 221).
template <typename T, int GRP, bool VEC>
__global__ void __launch_bounds__(256) i4_dequantize_kernel(const uint8_t* __restrict__ q, int64_t ldq,
                                                            const float* __restrict__ scale, int64_t lds, int64_t rows,
                                                            uint32_t pieces, T* __restrict__ w, int64_t ldw,
                                                            int64_t turns) {
  constexpr int N = 16 / sizeof(T), H = 8 / N;
  Place at(rows, pieces);
  for (int64_t turn = 0; turn < turns; ++turn) {
    int64_t row[UNROLL];
    uint32_t piece[UNROLL], c[UNROLL];
    float s[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      row[u] = at.row, piece[u] = at.at;
      at.next();
      if (row[u] >= rows) continue;
      const uint32_t word = piece[u] / H;
      c[u] = *reinterpret_cast<const uint32_t*>(q + row[u] * ldq + (int64_t)word * 4);
      s[u] = scale[row[u] * lds + word / (GRP / 8)];
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (row[u] >= rows) continue;
      const uint32_t code = c[u] >> (8 * (piece[u] % H));  // (codes 4 to 7 lie 8 bits above codes 0 to 3)
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = s[u] * (float)((int)((code >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15u) - 8);
      T* dst = w + row[u] * ldw + (int64_t)piece[u] * N;
      if constexpr (VEC && sizeof(T) == 4) {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(dst));
      } else if constexpr (VEC) {
        __builtin_nontemporal_store(u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])},
                                    reinterpret_cast<u32x4*>(dst));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) Elem<T>::st(dst, i, v[i]);
      }
    }
  }
}

// Workgroups for so many pieces (at most `cap`), and how often each takes UNROLL
// of them a thread.
void launch_size(int64_t pieces, int64_t cap, unsigned& grid, int64_t& turns) {
  grid = (unsigned)std::min<int64_t>(cdiv(pieces, 256 * UNROLL), cap);
  turns = cdiv(pieces, (int64_t)grid * 256 * UNROLL);
}

template <typename T, int GRP>
hipError_t quantize(const T* w, int64_t rows, int64_t cols, int64_t ldw, uint8_t* q, int64_t ldq, float* scale,
                    int64_t lds, hipStream_t s) {
  const uint32_t words = (uint32_t)(cols / 8), wpr = (uint32_t)(cdiv(cols, GRP) * (GRP / 8));
  unsigned grid;
  int64_t turns;
  launch_size(rows * wpr, (int64_t)num_cus() * 32, grid, turns);
  if (ldw % (int64_t)(16 / sizeof(T)) == 0)
    i4_quantize_kernel<T, GRP, true><<<grid, 256, 0, s>>>(w, rows, words, wpr, ldw, q, ldq, scale, lds, turns);
  else
    i4_quantize_kernel<T, GRP, false><<<grid, 256, 0, s>>>(w, rows, words, wpr, ldw, q, ldq, scale, lds, turns);
  return hipGetLastError();
}

template <typename T, int GRP>
hipError_t dequantize(const uint8_t* q, int64_t ldq, const float* scale, int64_t lds, int64_t rows, int64_t cols, T* w,
                      int64_t ldw, hipStream_t s) {
  const uint32_t pieces = (uint32_t)(cols / (16 / sizeof(T)));
  unsigned grid;
  int64_t turns;
  launch_size(rows * pieces, 1 << 23, grid, turns);  // (a launch has fewer than 2^32 threads)
  if (ldw % (int64_t)(16 / sizeof(T)) == 0)
    i4_dequantize_kernel<T, GRP, true><<<grid, 256, 0, s>>>(q, ldq, scale, lds, rows, pieces, w, ldw, turns);
  else
    i4_dequantize_kernel<T, GRP, false><<<grid, 256, 0, s>>>(q, ldq, scale, lds, rows, pieces, w, ldw, turns);
  return hipGetLastError();
}

// The linear layer: a workgroup computes RB rows x R channels over all of K, whose
// stretches of 256 its W waves take in turn (stream.h), each with one stage of
// LDS: the next stretch is copied while this one is multiplied.  More stages a
// wave cost workgroups of a CU, and were slower (one row, 6144 x 6144: 7.3 us
// with one stage, 8.0 with two; 64 rows, 3584 x 6144: 13.1 against 15.9 with four
// waves of two).
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

template <int GRP, int RB, int R, int W, typename OUT>
__global__ void __launch_bounds__(64 * W) i4_linear_kernel(LinearParams p) {
  using namespace stream;
  using ST = Stage<GRP, R, 1, false, RB>;
  static_assert(R % 16 == 0, "whole tiles: half of one would store its rows twice");
  constexpr int RED = W * RB * (R + 4) * 4;
  constexpr int RING = W * ST::BYTES;
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
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem) + wave * ST::BYTES;
  const uint8_t* stage = smem + wave * ST::BYTES;
  auto copy = [&](int k0) {
    ST::copy_w(src, k0, at, lane);
    ST::copy_x(src, xr, rows, k0, at, lane);
  };
  f32x4_t acc[ST::RT];
#pragma unroll
  for (int t = 0; t < ST::RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (wave * 256 < p.K) copy(wave * 256);
  for (int k0 = wave * 256; k0 < p.K; k0 += W * 256) {
    wait_vm<0>();
    asm volatile("" ::: "memory");
    ST st;
    st.read(stage, lane, ST::column(lane, RB));
    if (!ST::EARLY) st.multiply(acc, lane);
    reads_done();
    if (k0 + W * 256 < p.K) copy(k0 + W * 256);
    if (ST::EARLY) st.multiply(acc, lane);
  }
  // Partial sums [wave][row][channel] over the ring, once every wave is done with it.
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  const int col = lane & 15;
  if (col < RB) {
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

template <int GRP, int RB, int R, typename OUT>
hipError_t run_linear(LinearParams p, hipStream_t s) {
  constexpr int W = 8;
  p.mblocks = (int)cdiv(p.M, RB);
  p.ntiles = (int)cdiv(p.N, R);
  p.items = cdiv(p.ntiles, 8) * 8 * p.mblocks;
  const unsigned grid = (unsigned)std::min<int64_t>(p.items, 1 << 22);
  i4_linear_kernel<GRP, RB, R, W, OUT><<<grid, 64 * W, 0, s>>>(p);
  return hipGetLastError();
}

// Channels of a workgroup: 16 for up to four rows (one row, 6144 x 6144: 7.3 us, with
// 32 channels 7.9).  For more rows the fewest of 16, 32 and 64 that need no more
// workgroups than there are CUs, for each reads all of x: 16 rows, 6144 x 1792 5.4
// us with 32 channels (16: 7.8, 64: 6.6), 1024 x 2048 4.5 with 16 (32: 5.0); 64 rows,
// 3584 x 6144 13.1 with 64 (32: 16.4).
template <int GRP, typename OUT>
hipError_t linear(const LinearParams& p, hipStream_t s) {
  if (p.M == 1) return run_linear<GRP, 1, 16, OUT>(p, s);
  if (p.M <= 4) return run_linear<GRP, 4, 16, OUT>(p, s);
  const int64_t mblocks = cdiv(p.M, 16), cus = num_cus();
  if (cdiv(p.N, 16) * mblocks <= cus) return run_linear<GRP, 16, 16, OUT>(p, s);
  if (cdiv(p.N, 32) * mblocks <= cus) return run_linear<GRP, 16, 32, OUT>(p, s);
  return run_linear<GRP, 16, 64, OUT>(p, s);
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
