// lora_rotary.cuh — rotary positions outside the projection: tables for
// stretched contexts, and the rotation of finished q and k (or of their
// gradients) in layouts that the projection's epilogue (lora_norm_rope.cuh)
// does not cover: interleaved pairs, a rotated part of each head, any head
// size that is a multiple of 8.
//
//   (a, b) -> (a c - b s, b c + a s)     c, s = cos, sin of pair i at the token's position
//   half layout:        a = x[i], b = x[i + rot / 2]
//   interleaved layout: a = x[2 i], b = x[2 i + 1]
// The adjoint (the backward pass) turns by the opposite angle; tables that
// carry an amplitude scale both directions, as the transposed matrix does.
#pragma once

#include "lora_norm_rope.cuh"

namespace lora {

constexpr int kRotaryMaxPairs = 128;     // head_dim up to 256

// Turns per position of each pair, f_i / (2 pi): formed on the host in 64 bits.
struct RotaryTurns {
  double w[kRotaryMaxPairs];
};

// cos, sin [n_pos x pairs] fp32.  The angle of position p is p w turns; p w
// and its distance to the next whole turn are taken in 64 bits (an angle of
// 10^5 rad in 32 bits would be off by 4e-3), and the remainder, at most half
// a turn, is small enough for the 32-bit sincospi.  A thread keeps four pairs
// and walks over groups of four positions, 16 bytes of each table a step: the
// first position's angle that way, the next three by turning it on by w, 2 w
// and 3 w (two products and a sum each, within 3 * 2^-24 of the amplitude).
// 131072 x 64 pairs: 12.4 us (all four the first way, some 60 instructions a
// value: 16.0 us; the stores alone 10.4 us).
constexpr int kRotaryRun = 4;
constexpr int kRotaryTableCtas = 2;     // an SM: more repeat the three turns more often than they help the stores

__global__ void __launch_bounds__(256, kRotaryTableCtas)
    rotary_tables_kernel(const __grid_constant__ RotaryTurns turns, int pairs, long long n_pos, float amplitude,
                         float* __restrict__ cos_t, float* __restrict__ sin_t) {
  const int quads = pairs / 4;
  const int groups = blockDim.x / quads;            // of positions that a CTA is at
  const int q = threadIdx.x % quads;
  const double w[4] = {turns.w[4 * q], turns.w[4 * q + 1], turns.w[4 * q + 2], turns.w[4 * q + 3]};
  auto turn = [&](double t, float* s, float* c) { sincospif(2.0f * static_cast<float>(t - rint(t)), s, c); };
  grid_dep_wait();
  if (static_cast<int>(threadIdx.x) >= groups * quads) return;
  float dc[kRotaryRun - 1][4], ds[kRotaryRun - 1][4];
#pragma unroll
  for (int k = 1; k < kRotaryRun; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) turn(k * w[e], &ds[k - 1][e], &dc[k - 1][e]);
  for (long long p = (blockIdx.x * static_cast<long long>(groups) + threadIdx.x / quads) * kRotaryRun; p < n_pos;
       p += static_cast<long long>(gridDim.x) * groups * kRotaryRun) {
    float c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn(static_cast<double>(p) * w[e], &s[e], &c[e]);
      c[e] *= amplitude;
      s[e] *= amplitude;
    }
    float4* cp = reinterpret_cast<float4*>(cos_t + p * pairs) + q;
    float4* sp = reinterpret_cast<float4*>(sin_t + p * pairs) + q;
    *cp = make_float4(c[0], c[1], c[2], c[3]);
    *sp = make_float4(s[0], s[1], s[2], s[3]);
#pragma unroll
    for (int k = 0; k < kRotaryRun - 1; ++k) {
      if (p + k + 1 >= n_pos) break;
      cp += quads;
      sp += quads;
      float a[4], b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = fmaf(c[e], dc[k][e], -(s[e] * ds[k][e]));
        b[e] = fmaf(s[e], dc[k][e], c[e] * ds[k][e]);
      }
      *cp = make_float4(a[0], a[1], a[2], a[3]);
      *sp = make_float4(b[0], b[1], b[2], b[3]);
    }
  }
}

struct RotaryParams {
  const __nv_bfloat16* in[2];      // Q, K
  __nv_bfloat16* out[2];           // may be the inputs
  RopeTables t;                    // t.half = pairs of a head
  long long M;
  int heads[2];                    // of Q and of K (0: absent)
  int head_dim;
  int units;                       // 16-byte work units of a head: pair units, then copied chunks
  int slots;                       // threads that share a token's heads at one unit
  int interleaved;
  float sign;                      // of the sine: -1 for the adjoint
  uint32_t* status;
};

constexpr int kRotaryHeads = 4;    // heads a thread turns with the cosines it loaded

// One thread takes one unit (8 pairs: two 16-byte chunks) of up to
// kRotaryHeads heads of a token, so the table's 64 bytes are loaded once for
// them and all their data loads are in flight together.  Units past the
// rotated part copy one chunk (not launched when the rotation is in place).
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p) {
  grid_dep_wait();
  const long long idx = blockIdx.x * 256ll + threadIdx.x;
  const long long r = idx / p.units;
  const int u = static_cast<int>(idx - r * p.units);
  const long long m = r / p.slots;
  const int slot = static_cast<int>(r - m * p.slots);
  if (m >= p.M) return;
  const int pair_units = p.t.half / 8;
  const int heads = p.heads[0] + p.heads[1];
  const bool pairs = u < pair_units;
  int off_a, off_b;                                  // of the unit's chunks within a head
  if (!pairs) off_a = off_b = 2 * p.t.half + 8 * (u - pair_units);
  else if (p.interleaved) { off_a = 16 * u; off_b = off_a + 8; }
  else { off_a = 8 * u; off_b = off_a + p.t.half; }

  uint4 a[kRotaryHeads], b[kRotaryHeads];
  long long at[kRotaryHeads];
  int which[kRotaryHeads];
#pragma unroll
  for (int k = 0; k < kRotaryHeads; ++k) {
    const int h = slot + k * p.slots;
    which[k] = h >= p.heads[0];
    const int hh = which[k] ? h - p.heads[0] : h;
    at[k] = (m * p.heads[which[k]] + hh) * p.head_dim;
    if (h < heads) {
      a[k] = __ldcs(reinterpret_cast<const uint4*>(p.in[which[k]] + at[k] + off_a));
      if (pairs) b[k] = __ldcs(reinterpret_cast<const uint4*>(p.in[which[k]] + at[k] + off_b));
    }
  }
  const int pos = pairs ? p.t.pos[m] : 0;
  const bool outside = pos < 0 || pos >= p.t.n_pos;   // such a token passes through unturned
  if (!pairs || outside) {
    if (outside && pairs) atomicOr(p.status, kStatusBadArgument);
#pragma unroll
    for (int k = 0; k < kRotaryHeads; ++k) {
      if (slot + k * p.slots >= heads) break;
      *reinterpret_cast<uint4*>(p.out[which[k]] + at[k] + off_a) = a[k];
      if (pairs) *reinterpret_cast<uint4*>(p.out[which[k]] + at[k] + off_b) = b[k];
    }
    return;
  }
  float c[8], s[8];
  {
    const float4* cp = reinterpret_cast<const float4*>(p.t.cos + static_cast<long long>(pos) * p.t.half + 8 * u);
    const float4* sp = reinterpret_cast<const float4*>(p.t.sin + static_cast<long long>(pos) * p.t.half + 8 * u);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] *= p.sign;
  }
#pragma unroll
  for (int k = 0; k < kRotaryHeads; ++k) {
    if (slot + k * p.slots >= heads) break;
    float fa[8], fb[8], ya[8], yb[8];
    unpack_bf16x8(a[k], fa);
    unpack_bf16x8(b[k], fb);
    if (p.interleaved) {
      // chunk a holds pairs 0..3 of the unit, chunk b pairs 4..7
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ya[2 * e] = fa[2 * e] * c[e] - fa[2 * e + 1] * s[e];
        ya[2 * e + 1] = fa[2 * e + 1] * c[e] + fa[2 * e] * s[e];
        yb[2 * e] = fb[2 * e] * c[4 + e] - fb[2 * e + 1] * s[4 + e];
        yb[2 * e + 1] = fb[2 * e + 1] * c[4 + e] + fb[2 * e] * s[4 + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ya[e] = fa[e] * c[e] - fb[e] * s[e];
        yb[e] = fb[e] * c[e] + fa[e] * s[e];
      }
    }
    *reinterpret_cast<uint4*>(p.out[which[k]] + at[k] + off_a) = make_uint4(
        pack_bf16x2(ya[0], ya[1]), pack_bf16x2(ya[2], ya[3]), pack_bf16x2(ya[4], ya[5]), pack_bf16x2(ya[6], ya[7]));
    *reinterpret_cast<uint4*>(p.out[which[k]] + at[k] + off_b) = make_uint4(
        pack_bf16x2(yb[0], yb[1]), pack_bf16x2(yb[2], yb[3]), pack_bf16x2(yb[4], yb[5]), pack_bf16x2(yb[6], yb[7]));
  }
}

}  // namespace lora
