// Weights streamed through LDS to the matrix cores, for products of few rows:
// the pieces that the 4-bit linear layer and the decode step share.
//
// Such a product reads each weight once and is bound by HBM, so a wave keeps
// many loads in flight: it owns a ring of stages in LDS that it fills by LDS
// DMA, a stage holding the same stretch of k of R weight rows (channels) and of
// RB activation rows (tokens), and takes them in order, with no barrier: waves
// of a workgroup split k between them and add their sums at the end.
//
// Fragments are those of v_mfma_f32_16x16x32_bf16 with the channels as rows and
// the tokens as columns: lane l holds eight values of row l % 16 at k = 8 (l / 16),
// and of the result rows 4 (l / 16) .. + 3 of column l % 16.
//
// 4-bit codes q enter as the bf16 values 24 + q: a nibble n = q + 8 set into the
// upper four mantissa bits of 16 gives 16 + n, so that a word of eight codes becomes
// four registers by a shift and an and-or each.  The 24 times the sum of x that
// comes with it is taken off by products with a constant -24, whose sum the
// accumulator starts from.  All of it is exact but for the float32 sums, whose
// terms of an x are up to (24 + 31) |x| in place of 8 |x|: 3 bits of 24.
#pragma once

#include "gemm_dma.h"

namespace moe {
namespace stream {

using dma::dma16;
using dma::i32x4;
using dma::make_rsrc;
using dma::touch4u;
using dma::wait_vm;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// dma16 of bytes that are read once: they are the first to leave the L2, which
// keeps what is shared (activations, code).
__device__ __forceinline__ void dma16_once(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile(
      "s_nop 4\n\t"  // as in dma16
      "buffer_load_dwordx4 %0, %1, %2 offen nt lds"
      :
      : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds)
      : "memory");
}

constexpr uint32_t NOWHERE = 0x80000000u;  // an offset past every resource: the copy writes zeros

// The same resource in scalar registers (it is wave-uniform; kept across a loop
// it may have become a vector value, which a copy's operand cannot be).
__device__ __forceinline__ i32x4 scalar(i32x4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_readfirstlane(v[i]);
  return v;
}

// What a stage's copies read: the weights' rows (DUAL: of two matrices), their
// scales, the activations.  Bases may differ from tile to tile, pitches are in bytes.
struct Source {
  i32x4 w[2], s[2], x;
  uint32_t pitch, spitch;  // of a row of weights; of a row of scales
  int K, rows;             // k in all; rows of a part that exist
};

// GRP 0: bf16 weights; else 4 bits with a scale per GRP.  R weight rows (a
// multiple of 8; DUAL: eight of the first matrix, eight of the second, and so
// on) by SUB pieces of 128 bytes, RB activation rows.
template <int GRP, int R, int SUB, bool DUAL, int RB>
struct Stage {
  static constexpr bool I4 = GRP > 0;
  static constexpr int KC = I4 ? 256 : 64, KS = KC * SUB;  // k of a piece; of a stage
  static constexpr int PARTS = DUAL ? 2 : 1, PR = R / PARTS, RT = (R + 15) / 16;
  static constexpr int WB = R * SUB * 128, WI = WB / 1024;               // bytes; copies
  static constexpr int GPC = I4 ? KC / (I4 ? GRP : 1) : 0;               // groups of a stage
  static constexpr int SIP = (GPC * PR + 63) / 64, SI = SIP * PARTS, SB = SI * 256;
  static constexpr int XROW = KS * 2, XB = RB * XROW, XI = (XB + 1023) / 1024;  // (a row's pieces lie together)
  static constexpr int BYTES = WB + SB + XB;
  // (of a stage with room for that many activation rows)
  static constexpr __host__ __device__ int bytes(int rows) { return WB + SB + rows * XROW; }
  static constexpr int STEPS = SUB * KC / 32;  // products of 32 k
  // Whether a stage stays in registers while its slot is copied over, before it
  // is multiplied; else (too many) it is multiplied first.
  static constexpr bool EARLY = !I4 || (RT == 1 && GRP > 32);
  static_assert(!I4 || SUB == 1, "one piece of a 4-bit row per stage");
  static_assert(R % 8 == 0 && (!DUAL || R % 16 == 0), "rows");

  // LDS rows of weights are 128 bytes, 16-byte piece c of row r at c ^ (r & 6): the
  // 16 lanes that a ds_read_b128 serves at once then read from all banks.  The
  // activations' rows of 32 pieces (4 bits) keep piece 4 a + b of a half at
  // (4 b + a) ^ r for the same reason.
  static __device__ __forceinline__ int x_piece(int pos, int row) {
    if (!I4) return pos ^ (row & 6);
    const int p = (pos & 15) ^ (row & 15);
    return (pos & 16) | ((p & 3) << 2) | (p >> 2);
  }
  static __device__ __forceinline__ int x_pos(int piece, int row) {
    if (!I4) return piece ^ (row & 6);
    const int p = piece & 15;
    return (piece & 16) | ((((p & 3) << 2) | (p >> 2)) ^ (row & 15));
  }

  // Row of the activations that lane l's part of copy n belongs to.
  static __device__ __forceinline__ int x_row(int n, int lane) { return (n * 1024 + lane * 16) / XROW; }

  // Copies of the stage at k0 into LDS at `slot`: the weights and their scales.
  // A piece of a row that lies past K, or a row past `rows`, is not read.
  template <bool EDGE>
  static __device__ __forceinline__ void copy_w_as(const Source& s, int k0, uint32_t slot, int lane) {
    if (GRP == 32) asm volatile("" : "+v"(lane));  // (its many offsets computed here: kept over the loop they spill)
    const int r8 = lane >> 3, piece = ((lane & 7) ^ (r8 & 6)) * 16;
    const int at = I4 ? k0 / 2 : k0 * 2, left = (I4 ? (s.K / 2 + 15) & ~15 : s.K * 2) - at;  // bytes of the row from at on
    const i32x4 w[2] = {scalar(s.w[0]), DUAL ? scalar(s.w[1]) : i32x4{}};
    const uint32_t soff = __builtin_amdgcn_readfirstlane(at);
    const uint32_t v0 = __umul24(r8, s.pitch) + piece;  // (pitch < 2^24)
#pragma unroll
    for (int j = 0; j < WI; ++j) {
      const int sub = j / (R / 8), jr = j % (R / 8);
      const int part = DUAL ? jr & 1 : 0, row = (DUAL ? jr >> 1 : jr) * 8;
      uint32_t v = v0 + (uint32_t)row * s.pitch + (uint32_t)(sub * 128);
      if (EDGE) v = (int)(row + r8 >= s.rows) | (int)(sub * 128 + piece >= left) ? NOWHERE : v;
      dma16_once(w[part], v, soff, __builtin_amdgcn_readfirstlane(slot + j * 1024));
    }
    if constexpr (I4) {
      const int g0 = k0 / GRP, groups = (s.K + GRP - 1) / GRP - g0;  // (from g0 on)
      const uint32_t sat = __builtin_amdgcn_readfirstlane(g0 * 4);
#pragma unroll
      for (int n = 0; n < SIP; ++n) {
        const int i = n * 64 + lane, g = i / PR, row = i - g * PR;
        uint32_t v = __umul24(row, s.spitch) + (uint32_t)g * 4;
        if (EDGE) v = (int)(g >= groups) | (int)(row >= s.rows) ? NOWHERE : v;
        if (GPC * PR % 64 && n == SIP - 1) v = g >= GPC ? NOWHERE : v;
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          touch4u(scalar(s.s[p]), v, sat, __builtin_amdgcn_readfirstlane(slot + WB + (p * SIP + n) * 256));
      }
    }
  }
  static __device__ __forceinline__ void copy_w(const Source& s, int k0, uint32_t slot, int lane) {
    if (k0 + KS > s.K || s.rows < PR) copy_w_as<true>(s, k0, slot, lane);
    else copy_w_as<false>(s, k0, slot, lane);
  }

  // ... and the first `rows` (1 .. RB) rows of the activations; xr[n] is the byte
  // offset of row x_row(n, lane).  Zeros past K.  Returns the number of copies.
  static __device__ __forceinline__ int copy_x(const Source& s, const uint32_t (&xr)[XI], int rows, int k0,
                                               uint32_t slot, int lane) {
    const int bytes = rows * XROW;
    const i32x4 x = scalar(s.x);
    const uint32_t soff = __builtin_amdgcn_readfirstlane(k0 * 2);
#pragma unroll
    for (int n = 0; n < XI; ++n) {
      if (n * 1024 < bytes) {  // (uniform)
        const int byte = n * 1024 + lane * 16, row = x_row(n, lane), in = byte - row * XROW;
        const int k = (in / (KC * 2)) * KC + x_piece((in % (KC * 2)) / 16, row) * 8;
        const uint32_t v = k0 + k >= s.K ? NOWHERE : xr[n] + (uint32_t)k * 2;
        if (byte < bytes) dma16(x, v, soff, __builtin_amdgcn_readfirstlane(slot + WB + SB + n * 1024));
      }
    }
    return (bytes + 1023) / 1024;
  }

  // A stage in registers, and its products added to acc (rows 16 t + 4 (l / 16)
  // .. + 3, column l % 16; columns without a row repeat others or hold anything).
  bf16x8 b[STEPS];
  u32x4_t a[I4 ? 1 : STEPS][I4 ? 1 : RT];
  uint32_t c[I4 ? RT : 1][8];
  f32x4_t sc[I4 && EARLY ? GPC : 1][I4 && EARLY ? RT : 1];
  const uint8_t* from;

  // The scales of group g's result rows of tile t.
  __device__ __forceinline__ f32x4_t scale(int g, int t, int lane) const {
    const int q = lane >> 4, part = DUAL ? q >> 1 : 0;
    const int row = DUAL ? 8 * t + 4 * (q & 1) : 16 * t + 4 * (R - 16 * t < 16 ? q & 1 : q);
    return *reinterpret_cast<const f32x4_t*>(from + WB + part * SIP * 256 + (g * PR + row) * 4);
  }

  // The activation row that a lane reads, of a stage with room for `rows` (1 .. RB):
  // lanes past them read the last one, whose bytes the stage has.
  static __device__ __forceinline__ int column(int lane, int rows) {
    const int col = (lane & 15) % RB;
    return col < rows ? col : rows - 1;
  }

  // col: column(lane, rows), kept by the caller.
  __device__ __forceinline__ void read(const uint8_t* slot, int lane, int col) {
    const int r = lane & 15, q = lane >> 4;
    from = slot;
    auto xb = [&](int sub, int piece) {
      return *reinterpret_cast<const bf16x8*>(slot + WB + SB + col * XROW + sub * (KC * 2) + x_pos(piece, col) * 16);
    };
    if constexpr (!I4) {
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int sub = st / 2, ks = st % 2;
        b[st] = xb(sub, 4 * ks + q);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int row = 16 * t + (R - 16 * t < 16 ? r & 7 : r);  // (half a tile: its rows twice)
          a[st][t] = *reinterpret_cast<const u32x4_t*>(slot + (sub * R + row) * 128 + (((4 * ks + q) ^ (row & 6)) << 4));
        }
      }
    } else {
      constexpr int NJ = GRP / 32;  // words of a group that a lane holds
#pragma unroll
      for (int st = 0; st < 8; ++st) b[st] = xb(0, (st / NJ) * (4 * NJ) + q * NJ + st % NJ);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int row = 16 * t + (R - 16 * t < 16 ? r & 7 : r);  // (half a tile: its rows twice)
        const uint8_t* w = slot + row * 128;
        // A lane's words of group g; the part of the place that is the same in every row apart (an immediate offset).
        auto at = [&](int g) {
          const int word = g * 4 * NJ + q * NJ, low = NJ == 1 ? g & 1 : 0;
          return w + ((((word >> 2) - low) ^ (row & 6)) << 4) + (word & 3) * 4 + low * 16;
        };
#pragma unroll
        for (int g = 0; g < GPC; ++g) {
          if constexpr (NJ == 4) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at(g));
#pragma unroll
            for (int j = 0; j < 4; ++j) c[t][4 * g + j] = v[j];
          } else if constexpr (NJ == 2) {
            const u32x2_t v = *reinterpret_cast<const u32x2_t*>(at(g));
            c[t][2 * g] = v[0], c[t][2 * g + 1] = v[1];
          } else {
            c[t][g] = *reinterpret_cast<const uint32_t*>(at(g));
          }
          if constexpr (EARLY) sc[g][t] = scale(g, t, lane);
        }
      }
    }
  }

  // (mask and base are held in registers, so that each pair takes a shift and one bit-field insert)
  static __device__ __forceinline__ bf16x8 codes(uint32_t w, uint32_t mask, uint32_t base) {
    auto put = [&](uint32_t v) { return (v & mask) | (base & ~mask); };
    const u32x4_t v = {put(w << 3), put(w >> 1), put(w >> 5), put(w >> 9)};
    return __builtin_bit_cast(bf16x8, v);
  }

  __device__ __forceinline__ void multiply(f32x4_t (&acc)[RT], int lane) const {
    if constexpr (!I4) {
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[st][t]), b[st], acc[t], 0, 0, 0);
    } else {
      constexpr int NJ = GRP / 32;
      uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
      asm("" : "+s"(mask), "+v"(sixteen));
      const bf16x8 off = __builtin_bit_cast(bf16x8, u32x4_t{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u});  // -24
      // (a few independent chains side by side: a product's result is not ready for the next one's start)
      constexpr int GB = GPC < 4 ? GPC : RT > 1 ? 2 : 4;
#pragma unroll
      for (int g0 = 0; g0 < GPC; g0 += GB) {
        f32x4_t base[GB], p[GB][RT];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int g = 0; g < GB; ++g)
            base[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(off, b[(g0 + g) * NJ + j],
                                                              j ? base[g] : f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int g = 0; g < GB; ++g)
              p[g][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes(c[t][(g0 + g) * NJ + j], mask, sixteen), b[(g0 + g) * NJ + j],
                                                                j ? p[g][t] : base[g], 0, 0, 0);
#pragma unroll
        for (int g = 0; g < GB; ++g)
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            f32x4_t v;
            if constexpr (EARLY) v = sc[g0 + g][t];
            else v = scale(g0 + g, t, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] += v[i] * p[g][t][i];
          }
        if (!EARLY) __builtin_amdgcn_sched_barrier(0);  // (else the scales of all groups are held at once, and spill)
      }
    }
  }
};

// Waits until at most n copies (of those last asked for) are outstanding, or
// fewer: at once for n = COMMON, else for the next lower count that is coded.
template <int COMMON>
__device__ __forceinline__ void wait_younger(int n) {
  if (n == COMMON) wait_vm<COMMON>();
  else if (n >= 16) {
    if (n >= 24) n >= 32 ? wait_vm<32>() : n >= 28 ? wait_vm<28>() : wait_vm<24>();
    else n >= 21 ? wait_vm<21>() : n >= 18 ? wait_vm<18>() : wait_vm<16>();
  } else if (n >= 8) {
    if (n >= 12) n >= 14 ? wait_vm<14>() : wait_vm<12>();
    else n >= 10 ? wait_vm<10>() : wait_vm<8>();
  }
  else if (n >= 4) n >= 6 ? wait_vm<6>() : n >= 5 ? wait_vm<5>() : wait_vm<4>();
  else n >= 3 ? wait_vm<3>() : n >= 2 ? wait_vm<2>() : n >= 1 ? wait_vm<1>() : wait_vm<0>();
  asm volatile("" ::: "memory");
}

// Copies per stage of a ring, the oldest first, to know how many are younger than it.
struct Ages {
  uint64_t q = 0;
  int n = 0, sum = 0;
  __device__ __forceinline__ void push(int copies) {
    q |= (uint64_t)(uint32_t)copies << (8 * n);
    ++n;
    sum += copies;
  }
  __device__ __forceinline__ void pop() {  // sum is then of the younger ones
    sum -= (int)(q & 255);
    q >>= 8;
    --n;
  }
};

// LDS reads of a stage are complete before its slot is copied over.
__device__ __forceinline__ void reads_done() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

}  // namespace stream
}  // namespace moe
