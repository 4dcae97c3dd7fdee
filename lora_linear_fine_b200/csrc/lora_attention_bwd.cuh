// lora_attention_bwd.cuh — the attention backward on the tensor cores.
//
// Three launches, none of which adds to another's sums, so the order of every
// sum is fixed:
//   attn_delta_kernel  delta_i = do_i . o_i, and the row statistics by head
//   attn_dkv_kernel    a CTA a tile of 128 keys and a key / value head: dk, dv
//   attn_dq_kernel     a CTA a tile of 128 queries and a query head: dq
// The last two form p and ds each for itself: seven products a tile pair in
// place of five, against adding dq tiles into memory from every key tile,
// whose order would change from call to call and whose 64 KB a tile pair in
// fp32 would be more traffic than the two products take time.
#pragma once

#include "lora_attention.cuh"

namespace lora {

constexpr int kAttnBwdThreads = 384;     // warps: TMA, MMA, statistics, trimming, two warpgroups of elementwise work
constexpr int kAttnBwdPoly = 1;          // of four pairs of exponentials, those by the polynomial
constexpr int kAttnBwdRegsLow = 104, kAttnBwdRegsHigh = 200;

struct AttnBwdMaps {
  CUtensorMap q, k, v, d_o;   // [M x heads * D] bf16, box 64 x 128, 128-byte swizzle
};

// ---------------------------------------------------------------------------
// delta
// ---------------------------------------------------------------------------
// stat[0][h][m] = lse_mh log2(e), stat[1][h][m] = delta_mh.  A CTA takes 32
// rows of 8 heads; the results pass through shared memory so that both sides
// move whole sectors.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kLanes = D / 8, kPer = 256 / kLanes;      // threads a row and head; pairs of them at a time
  __shared__ float s[8][33];
  grid_dep_wait();
  const int m0 = blockIdx.x * 32, h0 = blockIdx.y * 8;
  const int lane = threadIdx.x % kLanes;
#pragma unroll
  for (int k = 0; k < 256 / kPer; ++k) {
    const int pair = k * kPer + threadIdx.x / kLanes;
    const int m = m0 + pair / 8, h = h0 + pair % 8;
    float d = 0.0f;
    if (m < p.M && h < p.heads) {
      const size_t at = (static_cast<size_t>(m) * p.heads + h) * D + 8 * lane;
      float a[8], b[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(p.dO + at), a);
      unpack_bf16x8(*reinterpret_cast<const uint4*>(p.O + at), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(a[e], b[e], d);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) s[pair % 8][pair / 8] = d;
  }
  __syncthreads();
  const int m = m0 + (threadIdx.x & 31), h = h0 + (threadIdx.x >> 5);
  if (m >= p.M || h >= p.heads) return;
  p.stat[static_cast<size_t>(h) * p.M + m] = p.lse[static_cast<size_t>(m) * p.heads + h] * kLog2e;
  p.stat[static_cast<size_t>(p.heads + h) * p.M + m] = s[threadIdx.x >> 5][threadIdx.x & 31];
}

// The A operand of dV, dK and dQ is written to tensor memory by two
// warpgroups, 64 columns of the tile each (the first one's 32 packed columns at
// `base`, the second one's at base + 64), in two parts of 32.  Part c of both
// is four steps of 16 out of the product's eight: k = 0 .. 3 -> step.
__device__ __forceinline__ int attn_part_step(int c, int k) { return (k / 2) * 4 + 2 * c + k % 2; }
__device__ __forceinline__ uint32_t attn_step_column(int kk) { return (kk / 4) * 64 + 8 * (kk % 4); }

// 64 columns of one warp's lanes to registers.
__device__ __forceinline__ void attn_ld64(uint32_t taddr, uint32_t (&v)[2][32]) {
  tmem_ld32(taddr, v[0]);
  tmem_ld32(taddr + 32, v[1]);
  tmem_wait_ld();
}

// ---------------------------------------------------------------------------
// dk, dv
// ---------------------------------------------------------------------------
// For each query head of the group and each query tile i that sees the keys
// (tiles transposed: rows are keys):
//   S = K Q_i^T, dP = V dO_i^T      both operands in shared memory
//   P = exp2(S - lse), dS = P (dP - delta)    256 threads, a row and 64 queries each
//   dV += P dO_i, dK += dS Q_i      P and dS read from tensor memory
// The products are issued as dV_i, S_i+1, dK_i, dP_i+1: while the elementwise
// work is at dS_i the tensor core does the first two, at P_i+1 the other two.
template <int D>
struct AttnDkvCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;         // of Q, and of dO
  static constexpr int kBars = 6 * kStages + 2 * kStages + 1 + 6 + 1;
  static constexpr int kSmemBytes = (2 + 2 * kStages) * kTileBytes + kStages * kAttnTile * 8 + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    attn_dkv_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnBwdMaps maps) {
  using C = AttnDkvCfg<D>;
  constexpr int T = kAttnTile, S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + C::kTileBytes;
  uint8_t* ring_q = sv + C::kTileBytes;
  uint8_t* ring_o = ring_q + S * C::kTileBytes;
  float* stat = reinterpret_cast<float*>(ring_o + S * C::kTileBytes);    // [S][2][T]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(stat + S * 2 * T);
  uint64_t* o_full = q_full + S;
  uint64_t* q_empty = o_full + S;
  uint64_t* o_empty = q_empty + S;
  uint64_t* q_land = o_empty + S;      // tiles that are trimmed before they count as full
  uint64_t* o_land = q_land + S;
  uint64_t* st_full = o_land + S;
  uint64_t* st_empty = st_full + S;
  uint64_t* kv_full = st_empty + S;
  uint64_t* s_full = kv_full + 1;
  uint64_t* p_full = s_full + 1;       // [2] quarters of P from both warpgroups
  uint64_t* dp_full = p_full + 2;
  uint64_t* ds_full = dp_full + 1;     // [2]
  uint64_t* mma_done = ds_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      for (uint64_t* b : {q_full, o_full, q_empty, o_empty, q_land, o_land, st_full}) mbar_init(&b[i], 1);
      mbar_init(&st_empty[i], 8);
    }
    mbar_init(kv_full, 1);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    for (int c = 0; c < 2; ++c) { mbar_init(&p_full[c], 8); mbar_init(&ds_full[c], 8); }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t tK = tbase, tV = tbase + D, tS = tbase + 256, tP = tbase + 384;
  grid_dep_wait();

  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(p.kv_heads);
  const int hk = static_cast<int>(blockIdx.x - tile * static_cast<uint32_t>(p.kv_heads));
  const bool live = attn_plan_ok(p) && tile < p.plan.head[kPlanKv];
  AttnTileRef t{0, 0, 0, 0};
  if (live) t = p.plan.kv[tile];
  const bool behind = t.prefix_end < 0;
  if (behind) {
    attn_zero_rows<D>(p.dK, p.kv_heads, hk, t.row0, min(t.row0 + T, t.end));
    attn_zero_rows<D>(p.dV, p.kv_heads, hk, t.row0, min(t.row0 + T, t.end));
  }
  // query tiles that see the keys: from the first one with a prefix, else from the keys' own
  const int group = p.heads / p.kv_heads;
  const int first = t.row0 < t.prefix_end ? t.begin : t.row0;
  const int n_tiles = (t.end - first + T - 1) / T;
  const int n = n_tiles * group;

  if (live && !behind && warp < 4) {
    regs_lower<kAttnBwdRegsLow>();
    if (warp == 0) {
      // -------------------------------------------------------------- TMA
      RingPos rq;
      bool ok = true;
      if (lane == 0) {
        mbar_arrive_expect_tx(kv_full, 2 * C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b) {
          tma_load_2d(sk + b * (T * 128), &maps.k, kv_full, hk * D + 64 * b, t.row0);
          tma_load_2d(sv + b * (T * 128), &maps.v, kv_full, hk * D + 64 * b, t.row0);
        }
        for (int i = 0; i < n && ok; ++i) {
          const int h = hk * group + i / n_tiles, row = first + (i % n_tiles) * T;
          const bool trim = row + T > t.end;
          for (int k = 0; k < 2 && ok; ++k) {
            ok = mbar_wait(k == 0 ? &q_empty[rq.stage] : &o_empty[rq.stage], rq.phase ^ 1u, ctl);
            if (!ok) break;
            uint64_t* bar = k == 0 ? (trim ? &q_land[rq.stage] : &q_full[rq.stage])
                                   : (trim ? &o_land[rq.stage] : &o_full[rq.stage]);
            uint8_t* dst = (k == 0 ? ring_q : ring_o) + rq.stage * C::kTileBytes;
            mbar_arrive_expect_tx(bar, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_2d(dst + b * (T * 128), k == 0 ? &maps.q : &maps.d_o, bar, h * D + 64 * b, row);
          }
          if (ok) rq.next(S);
        }
        if (!ok) {   // every copy has landed before the CTA may end
          mbar_wait(kv_full, 0, quiet);
          attn_drain(q_full, S, rq);
          attn_drain(o_full, S, rq);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA
      constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
      constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
      // A (keys, resident) times a ring tile's rows
      auto across = [&](uint64_t a, const uint8_t* ring, uint32_t stage, uint32_t d) {
        const uint64_t b = sdesc_sw128(smem_u32(ring), 16, 1024) + stage * (C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
            mma_bf16(d, a + off, b + off, kIdS, kk > 0);
          }
        }
      };
      // tensor memory (keys x queries) times a ring tile
      auto along = [&](uint32_t a, uint64_t* ready, uint32_t parity, const uint8_t* ring, uint32_t stage, uint32_t d,
                       bool fresh) {
        const uint64_t b = sdesc_sw128(smem_u32(ring), T * 128, 1024) + stage * (C::kTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!mbar_wait_warp(&ready[c], parity, ctl)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < T / 32; ++k) {
              const int kk = attn_part_step(c, k);
              mma_bf16_ta(d, a + attn_step_column(kk), b + kk * (2048 >> 4), kIdO, !fresh || c + k > 0);
            }
          }
        }
        return true;
      };
      const uint64_t k_desc = sdesc_sw128(smem_u32(sk), 16, 1024), v_desc = sdesc_sw128(smem_u32(sv), 16, 1024);
      RingPos r;
      bool ok = mbar_wait_warp(kv_full, 0, ctl) && mbar_wait_warp(&q_full[0], 0, ctl);
      if (ok) {
        tc_fence_after();
        across(k_desc, ring_q, 0, tS);
        if (elect_one()) mma_commit(s_full);
        ok = mbar_wait_warp(&o_full[0], 0, ctl);
      }
      if (ok) {
        tc_fence_after();
        across(v_desc, ring_o, 0, tP);
        if (elect_one()) mma_commit(dp_full);
      }
      for (int i = 0; i < n && ok; ++i) {
        RingPos nx = r;
        nx.next(S);
        ok = along(tS, p_full, i & 1, ring_o, r.stage, tV, i == 0);
        if (!ok) break;
        if (elect_one()) mma_commit(&o_empty[r.stage]);
        if (i + 1 < n) {
          ok = mbar_wait_warp(&q_full[nx.stage], nx.phase, ctl);
          if (!ok) break;
          tc_fence_after();
          across(k_desc, ring_q, nx.stage, tS);
          if (elect_one()) mma_commit(s_full);
        }
        ok = along(tP, ds_full, i & 1, ring_q, r.stage, tK, i == 0);
        if (!ok) break;
        if (elect_one()) mma_commit(&q_empty[r.stage]);
        if (i + 1 < n) {
          ok = mbar_wait_warp(&o_full[nx.stage], nx.phase, ctl);
          if (!ok) break;
          tc_fence_after();
          across(v_desc, ring_o, nx.stage, tP);
          if (elect_one()) mma_commit(dp_full);
        }
        r = nx;
      }
      if (elect_one()) mma_commit(mma_done);
      mbar_wait_warp(mma_done, 0, quiet);
    } else if (warp == 2) {
      // -------------------------------------------------------------- row statistics
      // Rows past the document: lse = infinity makes their p zero.
      RingPos r;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int h = hk * group + i / n_tiles, row = first + (i % n_tiles) * T;
        const float* a = p.stat + static_cast<size_t>(h) * p.M;
        const float* b = a + static_cast<size_t>(p.heads) * p.M;
        float l[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = row + e * 32 + lane;
          l[e] = m < t.end ? a[m] : INFINITY;
          d[e] = m < t.end ? b[m] : 0.0f;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&st_empty[r.stage], r.phase ^ 1u, ctl));
        if (!ok) break;
        float* s = stat + r.stage * 2 * T;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[e * 32 + lane] = l[e];
          s[T + e * 32 + lane] = d[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[r.stage]);
        r.next(S);
      }
    } else {
      // -------------------------------------------------------------- trimming
      // Rows past the document in its last query tile become zero: their p
      // and ds are zero, but zero times an infinity or NaN there would not be.
      RingPos r;
      uint32_t landed = 0;             // a bit a stage: parity of its next landing
      bool ok = (t.end - first) % T != 0;
      for (int i = 0; i < n && ok; ++i) {
        const int row = first + (i % n_tiles) * T;
        if (row + T > t.end) {
          for (int k = 0; k < 2 && ok; ++k) {
            ok = __all_sync(0xffffffffu, mbar_wait(k == 0 ? &q_land[r.stage] : &o_land[r.stage],
                                                   (landed >> r.stage) & 1u, ctl));
            if (!ok) break;
            attn_trim_tile<C::kBoxes>((k == 0 ? ring_q : ring_o) + r.stage * C::kTileBytes, t.end - row, lane);
            if (lane == 0) mbar_arrive(k == 0 ? &q_full[r.stage] : &o_full[r.stage]);
          }
          landed ^= 1u << r.stage;
        }
        r.next(S);
      }
    }
  } else if (live && !behind) {
    // ---------------------------------------------------------------- elementwise
    regs_raise<kAttnBwdRegsHigh>();
    const int half = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int key = t.row0 + (warp & 3) * 32 + lane;
    const uint32_t rS = tS + lanes + 64 * half, rP = tP + lanes + 64 * half;
    const bool all_keys = min(t.row0 + T, t.end) <= t.prefix_end;
    RingPos r;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const AttnScore<kCap, kBias> score(p, hk * group + i / n_tiles);
      const int i0 = first + (i % n_tiles) * T + 64 * half;          // the first of this thread's 64 queries
      ok = mbar_wait(&st_full[r.stage], r.phase, ctl) && mbar_wait(s_full, i & 1, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float* st = stat + r.stage * 2 * T + 64 * half;
      uint32_t v[2][32];
      float2 g[32];                     // p, then p d(cap tanh)
      attn_ld64(rS, v);
      score.template apply<2, true, true>(v, i0 - key, g);
      const float2 mul = both(score.mul);
      const bool part = !all_keys && i0 - 64 * half < t.row0 + T;
      const int lim = key < t.prefix_end ? 0 : key - i0;             // queries from this one on see the key
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = *reinterpret_cast<const float4*>(st + 32 * c + e);
          const float2 nl[2] = {make_float2(-l.x, -l.y), make_float2(-l.z, -l.w)};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = 16 * c + e / 2 + u;
            const float2 y = attn_exp2<kAttnBwdPoly>(fma2(pair_of(&v[c][e + 2 * u]), mul, nl[u]), i);
            AttnScore<kCap, kBias>::put(v[c], e + 2 * u, y);
          }
        }
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e < lim) v[c][e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 y = pair_of(&v[c][e]);
          w[e / 2] = pack_bf16x2(y.x, y.y);
          g[16 * c + e / 2] = kCap ? mul2(y, g[16 * c + e / 2]) : y;
        }
        tmem_st16(rS + 16 * c, w);
        attn_publish(&p_full[c], lane);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, i & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      attn_ld64(rP, v);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = *reinterpret_cast<const float4*>(st + T + 32 * c + e);
          const float2 a = mul2(g[16 * c + e / 2], add2(pair_of(&v[c][e]), make_float2(-d.x, -d.y)));
          const float2 b = mul2(g[16 * c + e / 2 + 1], add2(pair_of(&v[c][e + 2]), make_float2(-d.z, -d.w)));
          w[e / 2] = pack_bf16x2(a.x, a.y);
          w[e / 2 + 1] = pack_bf16x2(b.x, b.y);
        }
        tmem_st16(rP + 16 * c, w);
        attn_publish(&ds_full[c], lane);
      }
      if (lane == 0) mbar_arrive(&st_empty[r.stage]);
      r.next(S);
    }
    // the first warpgroup stores dk, the second dv
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(mma_done, 0, ctl));
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* out = (half == 0 ? p.dK : p.dV) + (static_cast<size_t>(key) * p.kv_heads + hk) * D;
      const float by = half == 0 ? p.scale : 1.0f;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32((half == 0 ? tK : tV) + lanes + c, o);
        tmem_wait_ld();
        if (key < t.end) attn_store32(out + c, o, by);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------
// For each key tile j that the queries see:
//   S = Q K_j^T, dP = dO V_j^T,  dS = exp2(S - lse) (dP - delta),  dQ += dS K_j
// S has two buffers (dS is written over the one it came from), so the products
// are issued as dP_j+1, dQ_j, S_j+2 and the exponentials of tile j + 1 need
// not wait for any of them.
template <int D>
struct AttnDqCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStagesK = D == 128 ? 3 : 4, kStagesV = D == 128 ? 2 : 4;
  static constexpr int kBars = 2 * kStagesK + 2 * kStagesV + 1 + 1 + 2 + 1 + 1 + 1;
  static constexpr int kSmemBytes = (2 + kStagesK + kStagesV) * kTileBytes + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    attn_dq_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnBwdMaps maps) {
  using C = AttnDqCfg<D>;
  constexpr int T = kAttnTile, SK = C::kStagesK, SV = C::kStagesV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* so = sq + C::kTileBytes;
  uint8_t* ring_k = so + C::kTileBytes;
  uint8_t* ring_v = ring_k + SK * C::kTileBytes;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(ring_v + SV * C::kTileBytes);
  uint64_t* k_empty = k_full + SK;
  uint64_t* v_full = k_empty + SK;
  uint64_t* v_empty = v_full + SV;
  uint64_t* qo_full = v_empty + SV;
  uint64_t* land = qo_full + 1;
  uint64_t* s_full = land + 1;         // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* mma_done = ds_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SK; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < SV; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); }
    mbar_init(qo_full, 1);
    mbar_init(land, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t tQ = tbase, tP = tbase + 128, tS = tbase + 256;
  grid_dep_wait();

  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(p.heads);
  const int h = static_cast<int>(blockIdx.x - tile * static_cast<uint32_t>(p.heads));
  const bool live = attn_plan_ok(p) && tile < p.plan.head[kPlanQ];
  AttnTileRef t{0, 0, 0, 0};
  if (live) t = p.plan.q[tile];
  const bool behind = t.prefix_end < 0;
  if (behind) attn_zero_rows<D>(p.dQ, p.heads, h, t.row0, min(t.row0 + T, t.end));
  const int hk = h / (p.heads / p.kv_heads);
  const int n = attn_key_tiles(t, t.row0, T);

  if (live && !behind && warp < 4) {
    regs_lower<kAttnBwdRegsLow>();
    if (warp == 0) {
      // -------------------------------------------------------------- TMA
      RingPos rk, rv;
      uint32_t landed = 0;
      bool ok = true;
      if (lane == 0) {
        mbar_arrive_expect_tx(qo_full, 2 * C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b) {
          tma_load_2d(sq + b * (T * 128), &maps.q, qo_full, h * D + 64 * b, t.row0);
          tma_load_2d(so + b * (T * 128), &maps.d_o, qo_full, h * D + 64 * b, t.row0);
        }
      }
      for (int j = 0; j < n && ok; ++j) {
        const int row = t.begin + j * T;
        // Rows past the document become zero (see the trimming in attn_dkv_kernel).
        const bool trim = row + T > t.end;
        for (int k = 0; k < 2 && ok; ++k) {
          RingPos& r = k == 0 ? rk : rv;
          ok = __all_sync(0xffffffffu, mbar_wait(k == 0 ? &k_empty[r.stage] : &v_empty[r.stage], r.phase ^ 1u, ctl));
          if (!ok) break;
          uint8_t* dst = (k == 0 ? ring_k : ring_v) + r.stage * C::kTileBytes;
          uint64_t* full = k == 0 ? &k_full[r.stage] : &v_full[r.stage];
          uint64_t* bar = trim ? land : full;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_2d(dst + b * (T * 128), k == 0 ? &maps.k : &maps.v, bar, hk * D + 64 * b, row);
          }
          if (trim) {
            ok = __all_sync(0xffffffffu, mbar_wait(land, landed & 1u, quiet));
            ++landed;
            attn_trim_tile<C::kBoxes>(dst, t.end - row, lane);
            if (lane == 0) mbar_arrive(full);
          }
          r.next(k == 0 ? SK : SV);
        }
      }
      if (lane == 0 && !ok) {
        mbar_wait(qo_full, 0, quiet);
        attn_drain(k_full, SK, rk);
        attn_drain(v_full, SV, rv);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA
      constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
      constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
      auto across = [&](const uint8_t* a, const uint8_t* ring, uint32_t stage, uint32_t d) {
        const uint64_t ad = sdesc_sw128(smem_u32(a), 16, 1024);
        const uint64_t b = sdesc_sw128(smem_u32(ring), 16, 1024) + stage * (C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
            mma_bf16(d, ad + off, b + off, kIdS, kk > 0);
          }
        }
      };
      RingPos ks, kd, v;             // K tiles of the scores, of dQ; V tiles
      auto scores = [&](int j) {
        if (!mbar_wait_warp(&k_full[ks.stage], ks.phase, ctl)) return false;
        tc_fence_after();
        across(sq, ring_k, ks.stage, tS + (j & 1) * T);
        if (elect_one()) mma_commit(&s_full[j & 1]);
        ks.next(SK);
        return true;
      };
      auto values = [&]() {
        if (!mbar_wait_warp(&v_full[v.stage], v.phase, ctl)) return false;
        tc_fence_after();
        across(so, ring_v, v.stage, tP);
        if (elect_one()) mma_commit(dp_full);
        if (elect_one()) mma_commit(&v_empty[v.stage]);
        v.next(SV);
        return true;
      };
      bool ok = mbar_wait_warp(qo_full, 0, ctl);
      ok = ok && scores(0) && values();
      if (n > 1) ok = ok && scores(1);
      for (int j = 0; j < n && ok; ++j) {
        ok = mbar_wait_warp(ds_full, j & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        if (j + 1 < n) ok = values();
        if (!ok) break;
        const uint64_t b = sdesc_sw128(smem_u32(ring_k), T * 128, 1024) + kd.stage * (C::kTileBytes >> 4);
        const uint32_t a = tS + (j & 1) * T;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < T / 16; ++kk)
            mma_bf16_ta(tQ, a + attn_step_column(kk), b + kk * (2048 >> 4), kIdO, j > 0 || kk > 0);
        }
        if (elect_one()) mma_commit(&k_empty[kd.stage]);
        kd.next(SK);
        if (j + 2 < n) ok = scores(j + 2);
      }
      if (elect_one()) mma_commit(mma_done);
      mbar_wait_warp(mma_done, 0, quiet);
    }
  } else if (live && !behind) {
    // ---------------------------------------------------------------- elementwise
    regs_raise<kAttnBwdRegsHigh>();
    const int half = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int row = t.row0 + (warp & 3) * 32 + lane;
    const bool mine = row < t.end;
    const int see = min(max(row + 1, t.prefix_end), t.end);              // keys [begin, see)
    const int all = min(max(t.row0 + 1, t.prefix_end), t.end);           // ... that every row sees
    const float lse2 = mine ? p.stat[static_cast<size_t>(h) * p.M + row] : INFINITY;
    const float delta = mine ? p.stat[static_cast<size_t>(p.heads + h) * p.M + row] : 0.0f;
    const AttnScore<kCap, kBias> score(p, h);
    const float2 mul = both(score.mul), shift = both(-lse2);
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      const int j0 = t.begin + j * T + 64 * half;                        // the first of this thread's 64 keys
      const uint32_t rS = tS + (j & 1) * T + lanes + 64 * half, rP = tP + lanes + 64 * half;
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j >> 1) & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[2][32];
      float2 g[32];                     // p d(cap tanh)
      attn_ld64(rS, v);
      score.template apply<2, true, true>(v, j0 - row, g);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int i = 16 * c + e / 2;
          const float2 y = attn_exp2<kAttnBwdPoly>(fma2(pair_of(&v[c][e]), mul, shift), i);
          g[i] = kCap ? mul2(y, g[i]) : y;
        }
      if (j0 + 64 > all) {
        const int lim = see - j0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (2 * i >= lim) g[i].x = 0.0f;
          if (2 * i + 1 >= lim) g[i].y = 0.0f;
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      attn_ld64(rP, v);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 y = mul2(g[16 * c + e / 2], add2(pair_of(&v[c][e]), both(-delta)));
          w[e / 2] = pack_bf16x2(y.x, y.y);
        }
        tmem_st16(rS + 16 * c, w);
      }
      attn_publish(ds_full, lane);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(mma_done, 0, ctl));
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* out = p.dQ + (static_cast<size_t>(row) * p.heads + h) * D + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t o[32];
        tmem_ld32(tQ + lanes + half * (D / 2) + c, o);
        tmem_wait_ld();
        if (mine) attn_store32(out + c, o, p.scale);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace lora
