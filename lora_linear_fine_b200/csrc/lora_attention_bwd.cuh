// lora_attention_bwd.cuh — the attention backward on the tensor cores.
//
// Two kernels, neither of which adds to another's sums, so the order of every
// sum is fixed:
//   attn_dq_kernel     items of 128 queries and a query head: delta, dq
//   attn_dkv_kernel    items of 128 keys and a key / value head: dk, dv
// Each forms p and ds for itself: seven products a tile pair in place of five,
// against adding dq tiles into memory from every key tile, whose order would
// change from call to call and whose 64 KB a tile pair in fp32 would be more
// traffic than the two products take time.
//
// delta_i = do_i . o_i comes from the rounded o, off by 2^-9 of |do| |o|, which
// is as much as dp - delta itself for rows that see a few keys.  So for rows
// whose keys all lie in one tile it is sum_j p_ij dp_ij in fp32, and a row that
// sees one key has ds = 0 exactly.  attn_dq_kernel leaves delta and lse by head
// for attn_dkv_kernel.  With a bias few keys count in long documents too: the
// sum is then formed on the way for dk, and dq takes ds in two bf16 parts
// (8192 tokens in 23 documents, cap and bias: dk off by 2.4e-3 of its norm
// instead of 2.7e-3, dq by 2.2e-3 instead of 2.7e-3; 87 us instead of 72).
#pragma once

#include "lora_attention.cuh"

namespace lora {

// Registers: 96 a thread at launch (the most for 640 threads), then 64 for the
// first four warps and 104 for the others.
constexpr int kAttnBwdRegsLow = 64, kAttnBwdRegsHigh = 104;
constexpr int kAttnBwdThreads = 640;     // warps: TMA, MMA, statistics, trimming, 16 of elementwise work

struct AttnBwdMaps {
  CUtensorMap q, k, v, d_o;   // [M x heads * D] bf16, box 64 x 128, 128-byte swizzle
};

// Part c of a thread's 32 packed values over its first columns.
template <int kParts>
__device__ __forceinline__ void attn_put_part(uint32_t taddr, int c, const uint32_t (&w)[16]) {
  if constexpr (kParts == 1) {
    tmem_st16(taddr, w);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = w[8 * c + i];
    tmem_st8(taddr + 8 * c, u);
  }
}

// ---------------------------------------------------------------------------
// dk, dv
// ---------------------------------------------------------------------------
// For each query head of the group and each query tile i that sees the keys
// (tiles transposed: rows are keys):
//   S = K Q_i^T, dP = V dO_i^T      both operands in shared memory
//   P = exp2(S - lse), dS = P (dP - delta)    512 threads, a row and 32 queries each
//   dV += P dO_i, dK += dS Q_i      P and dS read from tensor memory
// The products are issued as dV_i, S_i+1, dK_i, dP_i+1 (S_i+1 first where it
// has a buffer of its own): while the elementwise work is at dS_i the tensor
// core does the first two, at P_i+1 the other two.
//
// Few key tiles and heads leave SMs idle, or wait for the longest: then the
// steps of an item are cut into p.parts items that write fp32 sums, and
// attn_join_kernel adds these in order.
template <int D>
struct AttnDkvCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;         // of Q, and of dO
  static constexpr int kKv = D == 128 ? 1 : 2;             // of K and V
  // P and dS are handed over in two parts where the products take longer than
  // the elementwise work, so that they begin earlier; each hand-over costs the
  // warps some 100 cycles.
  static constexpr int kParts = D == 128 ? 2 : 1;
  // Buffers of S: with two the scores of the next tile are ready before this
  // one's work ends; with 128 features dk and dv leave room for one.
  static constexpr int kScores = D == 128 ? 1 : 2;
  static constexpr int kBars = 6 * kStages + 2 * kStages + 2 * kKv + 5 + kScores + 2 + 1;
  static constexpr int kSmemBytes = (2 * kKv + 2 * kStages) * kTileBytes + kStages * kAttnTile * 8 + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};

template <int D, AttnTanh kTanh, bool kBias>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    attn_dkv_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnBwdMaps maps) {
  using C = AttnDkvCfg<D>;
  constexpr bool kCap = kTanh != kNoCap;
  constexpr int T = kAttnTile, S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int NB = C::kKv, kParts = C::kParts, NS = C::kScores;
  uint8_t* sk = smem;                  // [NB]
  uint8_t* sv = sk + NB * C::kTileBytes;
  uint8_t* ring_q = sv + NB * C::kTileBytes;
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
  uint64_t* kv_full = st_empty + S;    // [NB]
  uint64_t* kv_empty = kv_full + NB;   // [NB]
  uint64_t* s_full = kv_empty + NB;    // [NS]
  // [NS][kParts]: a part of P from all warps.  One a buffer of S: with two of
  // them a warp may be at the next tile's P before another has finished this one's.
  uint64_t* p_full = s_full + NS;
  static_assert(NS * kParts == 2, "the barriers of P");
  uint64_t* dp_full = p_full + 2;
  uint64_t* ds_full = dp_full + 1;     // [2]
  uint64_t* acc_full = ds_full + 2;    // dk and dv of the item are complete
  uint64_t* acc_empty = acc_full + 1;  // ... and have been read
  uint64_t* mma_done = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      for (uint64_t* b : {q_full, o_full, q_empty, o_empty, q_land, o_land, st_full}) mbar_init(&b[i], 1);
      mbar_init(&st_empty[i], 16);
    }
    for (int i = 0; i < NB; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
    for (int i = 0; i < NS; ++i) mbar_init(&s_full[i], 1);
    mbar_init(dp_full, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 16);
    for (int c = 0; c < 2; ++c) { mbar_init(&p_full[c], 16); mbar_init(&ds_full[c], 16); }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t tK = tbase, tV = tbase + D, tS = tbase + 2 * D, tP = tbase + 2 * D + NS * T;
  grid_dep_wait();

  AttnItems items(p.plan.kv, attn_plan_ok(p) ? p.plan.head[kPlanKv] : 0u, p.kv_heads * p.parts);
  const int group = p.heads / p.kv_heads;
  bool ok = true;
  // The item's steps: query heads of the group times the query tiles that see
  // the keys (from the first one with a prefix, else from the keys' own), or
  // its share of them.
  struct Steps { int hk, part, first, n_tiles, n, h, row; };
  auto steps = [&] {
    Steps s;
    s.first = items.t.row0 < items.t.prefix_end ? items.t.begin : items.t.row0;
    s.n_tiles = (items.t.end - s.first + T - 1) / T;
    s.hk = items.h >> p.parts_log2;
    s.part = items.h & (p.parts - 1);
    s.n = s.n_tiles * group;
    s.h = s.hk * group;
    s.row = s.first;
    if (p.parts > 1) {       // few rows then: within 32 bits
      const int from = s.n * s.part >> p.parts_log2;
      s.n = (s.n * (s.part + 1) >> p.parts_log2) - from;
      const int g = from / s.n_tiles;
      s.h += g;
      s.row += (from - g * s.n_tiles) * T;
    }
    return s;
  };

  if (warp < 4) {
    regs_lower<kAttnBwdRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0) {
        RingPos rq;
        uint32_t turn = 0;
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const AttnTileRef t = items.t;
          const Steps st = steps();
          const int hk = st.hk, first = st.first;
          int h = st.h, row = st.row;
          for (int i = 0; i < st.n && ok; ++i) {
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
            if (!ok) break;
            rq.next(S);
            if (i == 0) {
              const uint32_t buf = turn % NB;
              ok = mbar_wait(&kv_empty[buf], ((turn / NB) & 1u) ^ 1u, ctl);
              if (!ok) break;
              ++turn;
              mbar_arrive_expect_tx(&kv_full[buf], 2 * C::kTileBytes);
              for (int b = 0; b < C::kBoxes; ++b) {
                tma_load_2d(sk + buf * C::kTileBytes + b * (T * 128), &maps.k, &kv_full[buf], hk * D + 64 * b, t.row0);
                tma_load_2d(sv + buf * C::kTileBytes + b * (T * 128), &maps.v, &kv_full[buf], hk * D + 64 * b, t.row0);
              }
            }
            row += T;
            if (row >= t.end) { row = first; ++h; }
          }
        }
        if (!ok) {   // every copy has landed before the CTA may end
          for (uint32_t k = turn > NB ? turn - NB : 0; k < turn; ++k) mbar_wait(&kv_full[k % NB], (k / NB) & 1u, quiet);
          attn_drain(q_full, S, rq);
          attn_drain(o_full, S, rq);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA
      if (elect_one()) {
        constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
        constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
        // a resident tile (keys) times a ring tile's rows
        auto across = [&](const uint8_t* res, uint32_t buf, const uint8_t* ring, uint32_t stage, uint32_t d, uint64_t* bar) {
          const uint64_t a = sdesc_sw128(smem_u32(res), 16, 1024) + buf * (C::kTileBytes >> 4);
          const uint64_t b = sdesc_sw128(smem_u32(ring), 16, 1024) + stage * (C::kTileBytes >> 4);
          {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
              mma_bf16(d, a + off, b + off, kIdS, kk > 0);
            }
            mma_commit(bar);
          }
        };
        // tensor memory (keys x queries) times a ring tile, which is free afterwards
        auto along = [&](uint32_t a, uint64_t* ready, uint32_t parity, const uint8_t* ring, uint32_t stage, uint32_t d,
                         bool fresh, uint64_t* bar) {
          const uint64_t b = sdesc_sw128(smem_u32(ring), T * 128, 1024) + stage * (C::kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < kParts; ++c) {
            if (!mbar_wait(&ready[c], parity, ctl)) return false;
            tc_fence_after();
            {
#pragma unroll
              for (int k = 0; k < T / 16 / kParts; ++k) {
                const int kk = kParts == 2 ? attn_part_step<32>(c, k) : k;
                mma_bf16_ta(d, a + attn_step_column<32>(kk), b + kk * (2048 >> 4), kIdO, !fresh || c + k > 0);
              }
              if (c == kParts - 1) mma_commit(bar);
            }
          }
          return true;
        };
        RingPos r;
        uint32_t turn = 0, step = 0;
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const int n = steps().n;
          if (n == 0) continue;
          const uint32_t buf = turn % NB;
          ok = mbar_wait(&kv_full[buf], (turn / NB) & 1u, ctl) && mbar_wait(&q_full[r.stage], r.phase, ctl);
          if (!ok) break;
          tc_fence_after();
          across(sk, buf, ring_q, r.stage, tS + step % NS * T, &s_full[step % NS]);
          ok = mbar_wait(&o_full[r.stage], r.phase, ctl);
          if (!ok) break;
          tc_fence_after();
          across(sv, buf, ring_o, r.stage, tP, dp_full);
          if (n == 1) mma_commit(&kv_empty[buf]);
          for (int i = 0; i < n && ok; ++i, ++step) {
            RingPos nx = r;
            nx.next(S);
            const uint32_t tA = tS + step % NS * T, next = (step + 1) % NS;
            auto next_scores = [&] {
              if (!mbar_wait(&q_full[nx.stage], nx.phase, ctl)) return false;
              tc_fence_after();
              across(sk, buf, ring_q, nx.stage, tS + next * T, &s_full[next]);
              return true;
            };
            if (NS == 2 && i + 1 < n) ok = next_scores();
            // the accumulators of the item before have been read
            if (i == 0) ok = ok && mbar_wait(acc_empty, (turn & 1u) ^ 1u, ctl);
            ok = ok && along(tA, p_full + step % NS * kParts, step / NS & 1u, ring_o, r.stage, tV, i == 0, &o_empty[r.stage]);
            if (NS == 1 && i + 1 < n) ok = ok && next_scores();
            ok = ok && along(tP, ds_full, step & 1u, ring_q, r.stage, tK, i == 0, &q_empty[r.stage]);
            if (!ok) break;
            if (i + 1 < n) {
              ok = mbar_wait(&o_full[nx.stage], nx.phase, ctl);
              if (!ok) break;
              tc_fence_after();
              across(sv, buf, ring_o, nx.stage, tP, dp_full);
              if (i + 2 == n) mma_commit(&kv_empty[buf]);
            }
            r = nx;
          }
          if (ok) mma_commit(acc_full);
          ++turn;
        }
        mma_commit(mma_done);
        mbar_wait(mma_done, 0, quiet);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------------- row statistics
      // Rows past the document: lse = infinity makes their p zero.
      RingPos r;
      while (ok && items.advance()) {
        if (items.behind()) continue;
        const AttnTileRef t = items.t;
        const Steps st = steps();
        const int first = st.first;
        int h = st.h, row = st.row;
        for (int i = 0; i < st.n && ok; ++i) {
          const float* a = p.stat + static_cast<size_t>(h) * p.M;
          const float* b = a + static_cast<size_t>(p.heads) * p.M;
          float l[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = row + e * 32 + lane;
            l[e] = m < t.end ? a[m] : -INFINITY;
            d[e] = m < t.end ? b[m] : 0.0f;
          }
          ok = mbar_wait_warp(&st_empty[r.stage], r.phase ^ 1u, ctl);
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
          row += T;
          if (row >= t.end) { row = first; ++h; }
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- trimming
      // Rows past the document in its last query tile become zero: their p and
      // ds are zero, but zero times an infinity or NaN there would not be.
      uint32_t slot = 0, landed = 0;     // ring slots so far; a bit a stage: parity of its next landing
      while (ok && items.advance()) {
        if (items.behind()) continue;
        const AttnTileRef t = items.t;
        const Steps st = steps();
        const int keep = (t.end - st.first) % T;
        // steps of the document's last query tile
        int i = (t.end - st.row + T - 1) / T - 1;
        for (; i < st.n && ok && keep != 0; i += st.n_tiles) {
          const uint32_t stage = (slot + i) % S;
          for (int k = 0; k < 2 && ok; ++k) {
            ok = mbar_wait_warp(k == 0 ? &q_land[stage] : &o_land[stage], (landed >> stage) & 1u, ctl);
            if (!ok) break;
            attn_trim_tile<C::kBoxes>((k == 0 ? ring_q : ring_o) + stage * C::kTileBytes, keep, lane);
            if (lane == 0) mbar_arrive(k == 0 ? &q_full[stage] : &o_full[stage]);
          }
          landed ^= 1u << stage;
        }
        slot += st.n;
      }
    }
  } else {
    // ---------------------------------------------------------------- elementwise
    regs_raise<kAttnBwdRegsHigh>();
    const int quarter = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t rP = tP + lanes + 32 * quarter;
    // sums of part `part` of the steps: of dk (before the scale), of dv
    auto part_of = [&](int part, int which) {
      return p.partial + static_cast<size_t>(2 * part + which) * p.M * p.kv_heads * D;
    };
    AttnScore<kTanh, kBias> score(p);
    const float2 mul = both(score.mul);
    RingPos r;
    uint32_t turn = 0, step = 0;
    while (ok && items.advance()) {
      const AttnTileRef t = items.t;
      if (items.behind()) {
        const int last = min(t.row0 + T, t.end), i = threadIdx.x - 128;
        const int hk = items.h >> p.parts_log2, part = items.h & (p.parts - 1);
        if (p.parts == 1) {
          attn_zero_rows<D>(p.dK, p.kv_heads, hk, t.row0, last, i, 512);
          attn_zero_rows<D>(p.dV, p.kv_heads, hk, t.row0, last, i, 512);
        } else {             // as many bytes as twice the features in bf16
          attn_zero_rows<2 * D>(reinterpret_cast<__nv_bfloat16*>(part_of(part, 0)), p.kv_heads, hk, t.row0, last, i, 512);
          attn_zero_rows<2 * D>(reinterpret_cast<__nv_bfloat16*>(part_of(part, 1)), p.kv_heads, hk, t.row0, last, i, 512);
        }
        continue;
      }
      const Steps sp = steps();
      const int hk = sp.hk, first = sp.first, n = sp.n;
      const int key = t.row0 + (warp & 3) * 32 + lane;
      const bool all_keys = min(t.row0 + T, t.end) <= t.prefix_end;
      int h = sp.h, tile0 = sp.row;
      if (n > 0) score.head(p, h);
      for (int i = 0; i < n && ok; ++i, ++step) {
        const int i0 = tile0 + 32 * quarter;                           // the first of this thread's 32 queries
        ok = mbar_wait_warp(&st_full[r.stage], r.phase, ctl) && mbar_wait_warp(&s_full[step % NS], step / NS & 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        const uint32_t rS = tS + step % NS * T + lanes + 32 * quarter;
        const float* st = stat + r.stage * 2 * T + 32 * quarter;
        uint32_t v[1][32];
        float2 g[16];                     // p, then p d(cap tanh)
        tmem_ld32(rS, v[0]);
        tmem_wait_ld();
        score.template values<true>(v[0], g);
        const float d0 = static_cast<float>(i0 - key);
        const bool part = !all_keys && tile0 < t.row0 + T;
        const int lim = key < t.prefix_end ? 0 : key - i0;             // queries from this one on see the key
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 l = *reinterpret_cast<const float4*>(st + e);   // -lse
          const float2 nl[2] = {make_float2(l.x, l.y), make_float2(l.z, l.w)};
#pragma unroll
          for (int u = 0; u < 2; ++u)
            AttnScore<kTanh, kBias>::put(
                v[0], e + 2 * u,
                attn_exp2<AttnScore<kTanh, kBias>::kPoly>(fma2(pair_of(&v[0][e + 2 * u]), mul, score.shifted(nl[u], d0, e + 2 * u, 1.0f)),
                                        e / 2 + u));
          if (e % (32 / kParts) == 32 / kParts - 4) {
            const int e0 = e + 4 - 32 / kParts;
            if (part) {
#pragma unroll
              for (int k = e0; k < e + 4; ++k)
                if (k < lim) v[0][k] = 0u;
            }
#pragma unroll
            for (int k = e0; k < e + 4; k += 2) {
              const float2 y = pair_of(&v[0][k]);
              w[k / 2] = pack_bf16x2(y.x, y.y);
              g[k / 2] = kCap ? mul2(y, g[k / 2]) : y;
            }
            attn_put_part<kParts>(rS, e0 / (32 / kParts), w);
            attn_publish(&p_full[step % NS * kParts + e0 / (32 / kParts)], lane);
          }
        }
        // the first row of a document without a longer prefix sees one key
        if (key == t.begin && i0 == t.begin && t.prefix_end <= t.begin + 1) g[0].x = 0.0f;
        ok = mbar_wait_warp(dp_full, step & 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(rP, v[0]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = *reinterpret_cast<const float4*>(st + T + e);   // -delta
          const float2 a = mul2(g[e / 2], add2(pair_of(&v[0][e]), make_float2(d.x, d.y)));
          const float2 b = mul2(g[e / 2 + 1], add2(pair_of(&v[0][e + 2]), make_float2(d.z, d.w)));
          w[e / 2] = pack_bf16x2(a.x, a.y);
          w[e / 2 + 1] = pack_bf16x2(b.x, b.y);
          if (e % (32 / kParts) == 32 / kParts - 4) {
            const int c = e / (32 / kParts);
            attn_put_part<kParts>(rP, c, w);
            attn_publish(&ds_full[c], lane);
          }
        }
        if (lane == 0) mbar_arrive(&st_empty[r.stage]);
        r.next(S);
        tile0 += T;
        if (tile0 >= t.end && i + 1 < n) { tile0 = first; score.head(p, ++h); }
      }
      if (n > 0) {
        ok = ok && mbar_wait_warp(acc_full, turn & 1u, ctl);
        if (!ok) break;
        ++turn;
        tc_fence_after();
      }
      // half of the warps store dk, half dv
      const bool is_k = quarter < 2;
      const int f0 = (quarter & 1) * (D / 2);
      const int key0 = key - lane;               // the warp's first
      const uint32_t acc = (is_k ? tK : tV) + lanes + f0;
      if (p.parts == 1) {
        const float by = is_k ? p.scale : 1.0f;
        uint4 w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 2; c += 32) {
          uint32_t o[32];
          tmem_ld32(acc + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 8) w[(c + e) / 8] = attn_pack8(&o[e], by);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
        const size_t stride = static_cast<size_t>(p.kv_heads) * D * 2;
        attn_store_rows<D / 16>(w, reinterpret_cast<uint8_t*>(is_k ? p.dK : p.dV) + key0 * stride +
                                       (static_cast<size_t>(hk) * D + f0) * 2, stride, t.end - key0, lane);
      } else {
        const size_t stride = static_cast<size_t>(p.kv_heads) * D * 4;
        uint8_t* out = reinterpret_cast<uint8_t*>(part_of(sp.part, is_k ? 0 : 1)) + key0 * stride +
                       (static_cast<size_t>(hk) * D + f0) * 4;
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
          uint32_t o[32] = {};
          if (n > 0) {
            tmem_ld32(acc + c, o);
            tmem_wait_ld();
          }
          uint4 w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          attn_store_rows<8>(w, out + c * 4, stride, t.end - key0, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (n > 0 && lane == 0) mbar_arrive(acc_empty);
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

// dk and dv from the sums of their parts, added in order.  y: dk, dv.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p) {
  grid_dep_wait();
  if (!attn_plan_ok(p) || p.plan.head[kPlanKv] == 0u) return;
  const size_t n = static_cast<size_t>(p.M) * p.kv_heads * D;
  const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const float* src = p.partial + blockIdx.y * n + i;
  float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
  for (int k = 1; k < p.parts; ++k) {
    const float4 c = *reinterpret_cast<const float4*>(src + 2 * k * n), d = *reinterpret_cast<const float4*>(src + 2 * k * n + 4);
    a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
    b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
  }
  const float by = blockIdx.y == 0 ? p.scale : 1.0f;
  *reinterpret_cast<uint4*>((blockIdx.y == 0 ? p.dK : p.dV) + i) =
      make_uint4(pack_bf16x2(a.x * by, a.y * by), pack_bf16x2(a.z * by, a.w * by), pack_bf16x2(b.x * by, b.y * by),
                 pack_bf16x2(b.z * by, b.w * by));
}

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------
// stat[0][h][m] = -lse_mh log2(e), stat[1][h][m] = -delta_mh are written here.
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
  static constexpr int kBars = 3 * kStagesK + 3 * kStagesV + 2 + 2 + 1 + 1 + 2 + 1;
  static constexpr int kSmemBytes = (2 + kStagesK + kStagesV) * kTileBytes + 3 * kAttnTile * 4 + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};

template <int D, AttnTanh kTanh, bool kBias>
__global__ void __launch_bounds__(kAttnBwdThreads, 1)
    attn_dq_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnBwdMaps maps) {
  using C = AttnDqCfg<D>;
  constexpr bool kCap = kTanh != kNoCap;
  constexpr int T = kAttnTile, SK = C::kStagesK, SV = C::kStagesV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = smem;
  uint8_t* so = sq + C::kTileBytes;
  uint8_t* ring_k = so + C::kTileBytes;
  uint8_t* ring_v = ring_k + SK * C::kTileBytes;
  float* share = reinterpret_cast<float*>(ring_v + SV * C::kTileBytes);      // [3][T]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(share + 3 * T);
  uint64_t* k_empty = k_full + SK;
  uint64_t* v_full = k_empty + SK;
  uint64_t* v_empty = v_full + SV;
  uint64_t* k_land = v_empty + SV;     // tiles that are trimmed before they count as full
  uint64_t* v_land = k_land + SK;
  uint64_t* qo_full = v_land + SV;
  uint64_t* qo_empty = qo_full + 1;
  uint64_t* s_full = qo_empty + 1;     // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;    // dq of the item is complete
  uint64_t* acc_empty = acc_full + 1;  // ... and has been read
  uint64_t* mma_done = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SK; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); mbar_init(&k_land[i], 1); }
    for (int i = 0; i < SV; ++i) { mbar_init(&v_full[i], 1); mbar_init(&v_empty[i], 1); mbar_init(&v_land[i], 1); }
    mbar_init(qo_full, 1);
    mbar_init(qo_empty, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4 * (D / 32));
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 16);
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

  AttnItems items(p.plan.q, attn_plan_ok(p) ? p.plan.head[kPlanQ] : 0u, p.heads);
  const int group = p.heads / p.kv_heads;
  bool ok = true;

  if (warp < 4) {
    regs_lower<kAttnBwdRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0) {
        RingPos rk, rv;
        uint32_t turn = 0;
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const AttnTileRef t = items.t;
          const int h = items.h, hk = h / group, n = attn_key_tiles(t, t.row0, T);
          for (int j = 0; j < n && ok; ++j) {
            const int row = t.begin + j * T;
            const bool trim = row + T > t.end;     // rows past the document become zero, as in attn_dkv_kernel
            for (int k = 0; k < 2 && ok; ++k) {
              RingPos& r = k == 0 ? rk : rv;
              ok = mbar_wait(k == 0 ? &k_empty[r.stage] : &v_empty[r.stage], r.phase ^ 1u, ctl);
              if (!ok) break;
              uint8_t* dst = (k == 0 ? ring_k : ring_v) + r.stage * C::kTileBytes;
              uint64_t* bar = k == 0 ? (trim ? &k_land[r.stage] : &k_full[r.stage])
                                     : (trim ? &v_land[r.stage] : &v_full[r.stage]);
              mbar_arrive_expect_tx(bar, C::kTileBytes);
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_2d(dst + b * (T * 128), k == 0 ? &maps.k : &maps.v, bar, hk * D + 64 * b, row);
              r.next(k == 0 ? SK : SV);
              if (j == 0 && k == 0) {
                ok = mbar_wait(qo_empty, (turn & 1u) ^ 1u, ctl);
                if (!ok) break;
                ++turn;
                mbar_arrive_expect_tx(qo_full, 2 * C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b) {
                  tma_load_2d(sq + b * (T * 128), &maps.q, qo_full, h * D + 64 * b, t.row0);
                  tma_load_2d(so + b * (T * 128), &maps.d_o, qo_full, h * D + 64 * b, t.row0);
                }
              }
            }
          }
        }
        if (!ok) {   // every copy has landed before the CTA may end
          mbar_wait(qo_full, (turn & 1u) ^ 1u, quiet);
          attn_drain(k_full, SK, rk);
          attn_drain(v_full, SV, rv);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA
      if (elect_one()) {
        constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
        constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
        auto across = [&](const uint8_t* res, const uint8_t* ring, uint32_t stage, uint32_t d, uint64_t* bar, uint64_t* bar2) {
          const uint64_t a = sdesc_sw128(smem_u32(res), 16, 1024);
          const uint64_t b = sdesc_sw128(smem_u32(ring), 16, 1024) + stage * (C::kTileBytes >> 4);
          {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
              mma_bf16(d, a + off, b + off, kIdS, kk > 0);
            }
            mma_commit(bar);
            if (bar2 != nullptr) mma_commit(bar2);
          }
        };
        RingPos ks, kd, v;             // K tiles of the scores, of dQ; V tiles
        uint32_t turn = 0, issued = 0, step = 0;      // items; score tiles issued; dS tiles taken
        auto scores = [&]() {
          if (!mbar_wait(&k_full[ks.stage], ks.phase, ctl)) return false;
          tc_fence_after();
          across(sq, ring_k, ks.stage, tS + (issued & 1u) * T, &s_full[issued & 1u], nullptr);
          ++issued;
          ks.next(SK);
          return true;
        };
        auto values = [&]() {
          if (!mbar_wait(&v_full[v.stage], v.phase, ctl)) return false;
          tc_fence_after();
          across(so, ring_v, v.stage, tP, dp_full, &v_empty[v.stage]);
          v.next(SV);
          return true;
        };
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const int n = attn_key_tiles(items.t, items.t.row0, T);
          ok = mbar_wait(qo_full, turn & 1u, ctl);
          ok = ok && scores() && values();
          if (n > 1) ok = ok && scores();
          if (ok && n == 1) mma_commit(qo_empty);
          // the accumulator of the item before has been read
          ok = ok && mbar_wait(acc_empty, (turn & 1u) ^ 1u, ctl);
          for (int j = 0; j < n && ok; ++j, ++step) {
            ok = mbar_wait(ds_full, step & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = sdesc_sw128(smem_u32(ring_k), T * 128, 1024) + kd.stage * (C::kTileBytes >> 4);
            if (j + 1 < n) {
              ok = values();
              if (!ok) break;
              if (j + 2 == n) mma_commit(qo_empty);       // the last use of Q and dO
            }
            const uint32_t a = tS + (step & 1u) * T;
            {
#pragma unroll
              for (int kk = 0; kk < T / 16; ++kk)
                mma_bf16_ta(tQ, a + attn_step_column<32>(kk), b + kk * (2048 >> 4), kIdO, j > 0 || kk > 0);
              if constexpr (kBias) {       // what bf16 leaves of dS
#pragma unroll
                for (int kk = 0; kk < T / 16; ++kk)
                  mma_bf16_ta(tQ, a + 16 + attn_step_column<32>(kk), b + kk * (2048 >> 4), kIdO, 1);
              }
              mma_commit(&k_empty[kd.stage]);
            }
            kd.next(SK);
            if (j + 2 < n) ok = scores();
          }
          if (ok) mma_commit(acc_full);
          ++turn;
        }
        mma_commit(mma_done);
        mbar_wait(mma_done, 0, quiet);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------------- trimming
      uint32_t slot = 0, k_landed = 0, v_landed = 0;
      while (ok && items.advance()) {
        if (items.behind()) continue;
        const AttnTileRef t = items.t;
        const int n = attn_key_tiles(t, t.row0, T), row = t.begin + (n - 1) * T;
        slot += n;
        if (row + T > t.end) {
          const uint32_t sk = (slot - 1) % SK, sv = (slot - 1) % SV;
          ok = mbar_wait_warp(&k_land[sk], (k_landed >> sk) & 1u, ctl);
          if (!ok) break;
          attn_trim_tile<C::kBoxes>(ring_k + sk * C::kTileBytes, t.end - row, lane);
          if (lane == 0) mbar_arrive(&k_full[sk]);
          ok = mbar_wait_warp(&v_land[sv], (v_landed >> sv) & 1u, ctl);
          if (!ok) break;
          attn_trim_tile<C::kBoxes>(ring_v + sv * C::kTileBytes, t.end - row, lane);
          if (lane == 0) mbar_arrive(&v_full[sv]);
          k_landed ^= 1u << sk;
          v_landed ^= 1u << sv;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- elementwise
    regs_raise<kAttnBwdRegsHigh>();
    const int quarter = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t rP = tP + lanes + 32 * quarter;
    AttnScore<kTanh, kBias> score(p);
    const float2 mul = both(score.mul);
    uint32_t turn = 0, step = 0;
    // A wait that gives up is one warp's answer (another may have looked a moment
    // later), and a warp that left for it would be missed at the barriers of
    // whole_row, which have no limit.  So it carries ok = false to the next of
    // them, whose answer all warps share: that one is the only way out.
    while (items.advance()) {
      const AttnTileRef t = items.t;
      const int h = items.h;
      if (items.behind()) {
        attn_zero_rows<D>(p.dQ, p.heads, h, t.row0, min(t.row0 + T, t.end), threadIdx.x - 128, 512);
        continue;
      }
      const int n = attn_key_tiles(t, t.row0, T);
      const int row = t.row0 + (warp & 3) * 32 + lane;
      const bool mine = row < t.end;
      const int see = min(max(row + 1, t.prefix_end), t.end);              // keys [begin, see)
      const int all = min(max(t.row0 + 1, t.prefix_end), t.end);           // ... that every row sees
      const float nlse = mine ? -p.lse[static_cast<size_t>(row) * p.heads + h] * kLog2e : -INFINITY;
      score.head(p, h);
      const float2 shift = both(nlse);
      const bool lone = see - t.begin == 1;
      // p of N keys from the products in v: all 32 of the thread at once, or, with
      // a cap, whose derivative takes registers too, 16
      constexpr int N = kCap || kBias ? 16 : 32;
      auto probabilities = [&](uint32_t (&v)[N], float2 (&y)[N / 2], float2 (&dt)[N / 2], int j0) {
        score.template values<true>(v, dt);
        const float d0 = static_cast<float>(j0 - row);
#pragma unroll
        for (int e = 0; e < N; e += 2)
          y[e / 2] = attn_exp2<AttnScore<kTanh, kBias>::kPoly>(
              fma2(pair_of(&v[e]), mul, score.shifted(shift, d0, e, 1.0f)), e / 2);
        if (j0 + N > all) {
          const int lim = see - j0;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            if (2 * i >= lim) y[i].x = 0.0f;
            if (2 * i + 1 >= lim) y[i].y = 0.0f;
          }
        }
      };
      // The four warps of a row add up; the first one's sum counts.
      const int r = (warp & 3) * 32 + lane;
      auto whole_row = [&](float part, bool good) {
        if (quarter > 0) share[(quarter - 1) * T + r] = part;
        if (!bar_sync_and<512>(1, good)) return false;
        if (quarter == 0) {
          const float delta = (part + share[r]) + (share[T + r] + share[2 * T + r]);
          share[r] = -delta;
          if (mine) p.stat[static_cast<size_t>(p.heads + h) * p.M + row] = -delta;
        }
        return bar_sync_and<512>(1, true);
      };
      // delta: a quarter of the row's terms here
      float sum = 0.0f;
      if (n == 1) {
        // sum_j p_ij dp_ij
        ok = ok && mbar_wait_warp(&s_full[step & 1u], (step >> 1) & 1u, ctl) && mbar_wait_warp(dp_full, step & 1u, ctl);
        if (ok) {
          tc_fence_after();
          float2 two = make_float2(0.0f, 0.0f);
#pragma unroll 1
          for (int c = 0; c < 32; c += N) {
            uint32_t v[N];
            float2 y[N / 2], dt[N / 2];
            tmem_ld(tS + (step & 1u) * T + lanes + 32 * quarter + c, v);
            tmem_wait_ld();
            probabilities(v, y, dt, t.begin + 32 * quarter + c);
            tmem_ld(rP + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < N; e += 2) two = fma2(y[e / 2], pair_of(&v[e]), two);
          }
          sum = two.x + two.y;
        }
      } else {
        // do_i . o_i: kL lanes a row, so that whole pieces of rows are read;
        // dO lies in shared memory until the item's second step at least
        constexpr int kL = D / 32;
        const int first = lane / kL * kL, chunk = quarter * kL + lane % kL, r0 = (warp & 3) * 32;
        uint4 o[kL];
#pragma unroll
        for (int i = 0; i < kL; ++i) {
          const int m = min(t.row0 + r0 + first + i, t.end - 1);
          o[i] = __ldg(reinterpret_cast<const uint4*>(p.O + (static_cast<size_t>(m) * p.heads + h) * D) + chunk);
        }
        ok = ok && mbar_wait_warp(qo_full, turn & 1u, ctl);
        if (ok) {
#pragma unroll
          for (int i = 0; i < kL; ++i) {
            const int r = r0 + first + i;
            const uint4 g = *reinterpret_cast<const uint4*>(so + (chunk / 8) * (T * 128) + r * 128 + ((chunk % 8) ^ (r & 7)) * 16);
            float2 two = mul2(unpack_bf16x2(o[i].x), unpack_bf16x2(g.x));
            two = fma2(unpack_bf16x2(o[i].y), unpack_bf16x2(g.y), two);
            two = fma2(unpack_bf16x2(o[i].z), unpack_bf16x2(g.z), two);
            two = fma2(unpack_bf16x2(o[i].w), unpack_bf16x2(g.w), two);
            float d = two.x + two.y;
#pragma unroll
            for (int k = 1; k < kL; k *= 2) d += __shfl_xor_sync(0xffffffffu, d, k);
            if (i == lane % kL) sum = d;
          }
        }
      }
      if (quarter == 0 && mine) p.stat[static_cast<size_t>(h) * p.M + row] = nlse;
      ok = whole_row(sum, ok);
      if (!ok) break;
      const float ndelta = share[r];
      float2 exact = make_float2(0.0f, 0.0f);      // sum_j p_ij dp_ij, for the dk / dv kernel
      for (int j = 0; j < n && ok; ++j, ++step) {
        const int j0 = t.begin + j * T + 32 * quarter;                     // the first of this thread's 32 keys
        const uint32_t rS = tS + (step & 1u) * T + lanes + 32 * quarter;
        ok = mbar_wait_warp(&s_full[step & 1u], (step >> 1) & 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        uint32_t low[32 / N][N / 2];
#pragma unroll
        for (int c = 0; c < 32 / N; ++c) {
          uint32_t v[N], w[N / 2];
          float2 y[N / 2], dt[N / 2];
          tmem_ld(rS + N * c, v);
          tmem_wait_ld();
          probabilities(v, y, dt, j0 + N * c);
#pragma unroll
          for (int i = 0; i < N / 2; ++i)
            if (lone) y[i] = make_float2(0.0f, 0.0f);
          if (c == 0) {
            ok = mbar_wait_warp(dp_full, step & 1u, ctl);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_ld(rP + N * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const float2 dp = pair_of(&v[e]);
            if constexpr (kBias) exact = fma2(y[e / 2], dp, exact);
            float2 ds = mul2(y[e / 2], add2(dp, both(ndelta)));
            if constexpr (kCap) ds = mul2(ds, dt[e / 2]);
            w[e / 2] = pack_bf16x2(ds.x, ds.y);
            if constexpr (kBias) {
              const float2 rest = fma2(unpack_bf16x2(w[e / 2]), both(-1.0f), ds);
              low[c][e / 2] = pack_bf16x2(rest.x, rest.y);
            }
          }
          tmem_st(rS + N / 2 * c, w);           // over columns that this warp has read
        }
        if constexpr (kBias) {
#pragma unroll
          for (int c = 0; c < 32 / N; ++c) tmem_st(rS + 16 + N / 2 * c, low[c]);
        }
        if (!ok) break;
        attn_publish(ds_full, lane);
      }
      if (kBias && n > 1) ok = whole_row(exact.x + exact.y, ok);
      ok = ok && mbar_wait_warp(acc_full, turn & 1u, ctl);
      if (!ok) continue;
      ++turn;
      tc_fence_after();
      // 64-byte pieces of a row: by all warps, or by the first half of them
      constexpr int kPieces = D / 32;
      if (quarter < kPieces) {
        uint32_t o[32];
        tmem_ld32(tQ + lanes + 32 * quarter, o);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
        uint4 w[4];
#pragma unroll
        for (int e = 0; e < 32; e += 8) w[e / 8] = attn_pack8(&o[e], p.scale);
        const int row0 = row - lane;
        const size_t stride = static_cast<size_t>(p.heads) * D * 2;
        attn_store_rows<4>(w, reinterpret_cast<uint8_t*>(p.dQ) + row0 * stride +
                                  (static_cast<size_t>(h) * D + 32 * quarter) * 2, stride, t.end - row0, lane);
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
