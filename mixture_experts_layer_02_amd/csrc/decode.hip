// The whole expert layer for a few tokens (T <= 64).
#include <algorithm>

#include "internal.h"

namespace moe {

namespace {

// A row's words of eight weights as float: bf16, or 4 bits with a scale per GRP.
template <int GRP>
struct Weights {
  const uint8_t* q;
  const float* s;
  __device__ __forceinline__ void load(int64_t row, int words, int word, float (&v)[8]) const {
    if (GRP == 0) {
      Vec16<uint16_t>::load(reinterpret_cast<const uint16_t*>(q) + (row * words + word) * 8, v);
    } else {
      constexpr int L = GRP ? GRP / 8 : 1;
      const uint32_t c = reinterpret_cast<const uint32_t*>(q)[row * words + word];
      const float sc = s[row * ((words + L - 1) / L) + word / L];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sc * (float)((int)((c >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15u) - 8);
    }
  }
};

template <int GRP>
__device__ __forceinline__ float dot(const Weights<GRP>& w, int64_t row, const uint16_t* x, int words, int lane) {
  float sum = 0.f;
  for (int word = lane; word < words; word += 64) {
    float a[8], b[8];
    w.load(row, words, word, a);
    Vec16<uint16_t>::load(x + (int64_t)word * 8, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += a[j] * b[j];
  }
  return wave_sum(sum);
}

// One wave per token and expert.
__global__ void __launch_bounds__(256) logits_kernel(int T, int d, int E, const uint16_t* x, const uint16_t* wr,
                                                     const float* bias, float* logits) {
  const int i = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (i >= T * E) return;
  const Weights<0> w{reinterpret_cast<const uint8_t*>(wr), nullptr};
  const float v = dot(w, i % E, x + (int64_t)(i / E) * d, d / 8, lane);
  if (lane == 0) logits[i] = v + (bias ? bias[i % E] : 0.f);
}

// One wave per slot and channel of f: h[slot] = silu(G) U.
template <int GRP>
__global__ void __launch_bounds__(256) gate_up_kernel(moe_desc D, const uint16_t* x, const int32_t* idx,
                                                      Weights<GRP> w1, Weights<GRP> w3, uint16_t* h) {
  const int lane = threadIdx.x & 63;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < (int64_t)D.T * D.k * D.f; i += (int64_t)gridDim.x * 4) {
    const int64_t slot = i / D.f, n = i % D.f;
    const int e = idx[slot] - D.expert_begin;
    if (e < 0 || e >= D.num_local) continue;
    const uint16_t* xr = x + (slot / D.k) * D.d;
    const float g = dot(w1, (int64_t)e * D.f + n, xr, D.d / 8, lane);
    const float u = dot(w3, (int64_t)e * D.f + n, xr, D.d / 8, lane);
    if (lane == 0) h[i] = f2bf(g * sigmoidf_(g) * u);
  }
}

// One wave per token and channel of d.
template <int GRP>
__global__ void __launch_bounds__(256) down_kernel(moe_desc D, const uint16_t* h, const int32_t* idx, const float* w,
                                                   Weights<GRP> w2, uint16_t* y) {
  const int lane = threadIdx.x & 63;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < (int64_t)D.T * D.d; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / D.d, n = i % D.d;
    float sum = 0.f;
    for (int j = 0; j < D.k; ++j) {
      const int64_t slot = t * D.k + j;
      const int e = idx[slot] - D.expert_begin;
      if (e < 0 || e >= D.num_local) continue;
      sum += w[slot] * dot(w2, (int64_t)e * D.d + n, h + slot * D.f, D.f / 8, lane);
    }
    if (lane == 0) y[i] = f2bf(sum);
  }
}

size_t logits_bytes(const moe_desc& d) { return ((size_t)d.T * d.E * 4 + 255) / 256 * 256; }

template <int GRP>
hipError_t decode(const moe_desc& d, const void* x, const void* w1, const float* s1, const void* w3, const float* s3,
                  const void* w2, const float* s2, const int32_t* idx, const float* w, void* y, void* ws, hipStream_t s) {
  uint16_t* h = reinterpret_cast<uint16_t*>((char*)ws + logits_bytes(d));
  auto grid = [](int64_t waves) { return (unsigned)std::min<int64_t>((waves + 3) / 4, (int64_t)num_cus() * 64); };
  const Weights<GRP> a{(const uint8_t*)w1, s1}, b{(const uint8_t*)w3, s3}, c{(const uint8_t*)w2, s2};
  gate_up_kernel<GRP><<<grid((int64_t)d.T * d.k * d.f), 256, 0, s>>>(d, (const uint16_t*)x, idx, a, b, h);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  down_kernel<GRP><<<grid((int64_t)d.T * d.d), 256, 0, s>>>(d, h, idx, w, c, (uint16_t*)y);
  return hipGetLastError();
}

}  // namespace

size_t decode_workspace(const moe_desc& d) { return logits_bytes(d) + (size_t)d.T * d.k * d.f * 2; }

hipError_t launch_decode(const moe_desc& d, int group, int n_groups, const void* x, const void* Wr, const float* bias,
                         const void* W1, const float* W1s, const void* W3, const float* W3s, const void* W2,
                         const float* W2s, int32_t* idx, float* w, void* y, void* ws, hipStream_t s) {
  if (Wr) {
    float* logits = reinterpret_cast<float*>(ws);
    logits_kernel<<<(d.T * d.E + 3) / 4, 256, 0, s>>>(d.T, d.d, d.E, (const uint16_t*)x, (const uint16_t*)Wr, bias, logits);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_route(d, logits, n_groups, idx, w, s);
    if (e != hipSuccess) return e;
  }
  switch (group) {
    case 0: return decode<0>(d, x, W1, W1s, W3, W3s, W2, W2s, idx, w, y, ws, s);
    case 32: return decode<32>(d, x, W1, W1s, W3, W3s, W2, W2s, idx, w, y, ws, s);
    case 64: return decode<64>(d, x, W1, W1s, W3, W3s, W2, W2s, idx, w, y, ws, s);
    default: return decode<128>(d, x, W1, W1s, W3, W3s, W2, W2s, idx, w, y, ws, s);
  }
}

}  // namespace moe
