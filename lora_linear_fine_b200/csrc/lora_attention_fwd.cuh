// lora_attention_fwd.cuh — the attention forward on the tensor cores.
//
// A CTA takes up to 256 query rows of one document and one head: two tiles of
// 128 rows, a and b, that share the key / value tiles of 128 rows.  For each
// key tile j and each of a, b:
//   S = Q K_j^T          tcgen05.mma, both operands in shared memory, S in tensor memory
//   P = exp2(z - m)      a warpgroup, one thread a row: S to registers, bf16 P back over S
//   O += P V_j           tcgen05.mma with P read from tensor memory
// so the scores never leave the SM.  While one warpgroup works on its S the
// tensor core works for the other one.  Tensor memory: S a, S b (128 columns
// each, P over their first 64), O a, O b.
//
// The running maximum m is only followed when a row's scores outgrow it by
// more than 2^8: until then P and the row's sum l are both larger by the same
// factor, at most 2^8, which fp32 and bf16 hold as well; the rescaling of O in
// tensor memory (a read and a write of all of it) becomes rare.  P is rounded
// to bf16 for the tensor core; l adds the fp32 values.
#pragma once

#include "lora_attention.cuh"

namespace lora {

template <int D>
struct AttnFwdCfg {
  static constexpr int kBoxes = D / 64;                          // 128-byte column boxes of a tile
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;               // K and V tiles in flight
  static constexpr int kBars = 2 * kStages + 1 + 1 + 2 + 4 + 2 + 1;
  static constexpr int kSmemBytes = (2 + kStages) * kTileBytes + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};
// Registers: 168 a thread at launch (the most for 384 threads), then 104 for
// the first warpgroup and 200 for the softmax ones, whose row of 128 scores
// stays in registers.
constexpr int kAttnFwdRegsLow = 104, kAttnFwdRegsHigh = 200;
constexpr int kAttnFwdPoly = 1;          // of four pairs of exponentials, those by the polynomial
constexpr int kAttnFwdThreads = 384;     // warps: TMA, MMA, two idle, softmax of tile a (4), of tile b (4)

struct AttnFwdMaps {
  CUtensorMap q, k, v;     // [M x heads * D] bf16, box 64 x 128, 128-byte swizzle
};

template <int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kAttnFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnFwdMaps maps) {
  using C = AttnFwdCfg<D>;
  constexpr int T = kAttnTile, S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * C::kTileBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * C::kTileBytes);
  uint64_t* empty = full + S;
  uint64_t* q_full = empty + S;
  uint64_t* land = q_full + 1;       // a tile that is trimmed before it counts as full
  uint64_t* s_full = land + 1;       // [2] S of this key tile is in tensor memory
  uint64_t* p_full = s_full + 2;     // [2][2] that half of P is in tensor memory (and O rescaled)
  uint64_t* pv_done = p_full + 4;    // [2] O holds this key tile
  uint64_t* mma_done = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(q_full, 1);
    mbar_init(land, 1);
    for (int x = 0; x < 2; ++x) { mbar_init(&s_full[x], 1); mbar_init(&p_full[2 * x], 4); mbar_init(&p_full[2 * x + 1], 4); mbar_init(&pv_done[x], 1); }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (threadIdx.x / 32 == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // Tensor memory is held before a dependent kernel may start (grid_dep_wait),
  // so none of its CTAs can take what a CTA of this grid still waits for.
  grid_dep_wait();

  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(p.heads);
  const int h = static_cast<int>(blockIdx.x - tile * static_cast<uint32_t>(p.heads));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool live = attn_plan_ok(p) && tile < p.plan.head[kPlanFwd];
  AttnTileRef t{0, 0, 0, 0};       // no rows: every role below has nothing to do
  if (live) t = p.plan.fwd[tile];
  const bool behind = t.prefix_end < 0;
  if (behind) {
    attn_zero_rows<D>(p.O, p.heads, h, t.row0, min(t.row0 + 2 * T, t.end));
    for (int r = t.row0 + static_cast<int>(threadIdx.x); r < min(t.row0 + 2 * T, t.end); r += kAttnFwdThreads)
      p.lse[static_cast<size_t>(r) * p.heads + h] = -INFINITY;
  }

  const int hk = h / (p.heads / p.kv_heads);
  const int tiles_x = t.row0 + T < t.end ? 2 : 1;
  // key tiles that the rows of tile x see
  const int n_a = attn_key_tiles(t, t.row0, T), n = tiles_x == 2 ? attn_key_tiles(t, t.row0 + T, T) : n_a;

  if (live && !behind && warp < 4) {
    regs_lower<kAttnFwdRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA
      RingPos rp;
      uint32_t issued = 0, landed = 0;
      bool ok = true;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tiles_x * C::kTileBytes));
        for (int x = 0; x < tiles_x; ++x)
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_2d(smem + x * C::kTileBytes + b * (T * 128), &maps.q, q_full, h * D + 64 * b, t.row0 + x * T);
      }
      for (int j = 0; j < n && ok; ++j)
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int row = t.begin + j * T;
          uint8_t* dst = ring + rp.stage * C::kTileBytes;
          ok = mbar_wait(&empty[rp.stage], rp.phase ^ 1u, ctl);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // Rows past the document in its last value tile are zeroed: their P
          // is zero, but zero times an infinity or NaN there would not be.
          const bool trim = kv == 1 && row + T > t.end;
          uint64_t* bar = trim ? land : &full[rp.stage];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_2d(dst + b * (T * 128), kv == 0 ? &maps.k : &maps.v, bar, hk * D + 64 * b, row);
          }
          if (trim) {
            ok = __all_sync(0xffffffffu, mbar_wait(land, landed & 1u, quiet));
            ++landed;
            attn_trim_tile<C::kBoxes>(dst, t.end - row, lane);
            if (lane == 0) mbar_arrive(&full[rp.stage]);
          } else {
            ++issued;
          }
          rp.next(S);
        }
      // Every copy has landed before the CTA may end.
      if (lane == 0 && !ok) {
        mbar_wait(q_full, 0, quiet);
        attn_drain(full, S, rp);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
      constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(ring), T * 128, 1024);
      auto scores = [&](int x, uint32_t stage) {
        const uint64_t a = q_desc + x * (C::kTileBytes >> 4), b = k_desc + stage * (C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
            mma_bf16(tbase + x * T, a + off, b + off, kIdS, kk > 0);
          }
        }
        if (elect_one()) mma_commit(&s_full[x]);
      };
      // half of the keys: 4 steps of 16
      auto values = [&](int x, uint32_t stage, int half, bool first) {
        const uint64_t b = v_desc + stage * (C::kTileBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < T / 32; ++k) {
            const int kk = half * (T / 32) + k;
            mma_bf16_ta(tbase + 256 + x * T, tbase + x * T + 8 * kk, b + kk * (2048 >> 4), kIdO, !first || kk > 0);
          }
        }
      };
      RingPos rp;
      bool ok = mbar_wait_warp(q_full, 0, ctl) && mbar_wait_warp(&full[0], 0, ctl);
      tc_fence_after();
      if (ok) {
        for (int x = 0; x < tiles_x; ++x) scores(x, 0);
        if (elect_one()) mma_commit(&empty[0]);
        rp.next(S);
      }
      for (int j = 0; j < n && ok; ++j) {
        const RingPos v = rp;
        ok = mbar_wait_warp(&full[v.stage], v.phase, ctl);
        rp.next(S);
        const RingPos k = rp;
        if (ok && j + 1 < n) {
          ok = mbar_wait_warp(&full[k.stage], k.phase, ctl);
          rp.next(S);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int nx = x == 0 ? n_a : (tiles_x == 2 ? n : 0);
          if (!ok || j >= nx) continue;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && mbar_wait_warp(&p_full[2 * x + half], j & 1, ctl);
            if (!ok) break;
            tc_fence_after();
            values(x, v.stage, half, j == 0);
          }
          if (!ok) continue;
          if (elect_one()) mma_commit(&pv_done[x]);
          if (j + 1 < nx) scores(x, k.stage);
        }
        if (ok) {
          if (elect_one()) mma_commit(&empty[v.stage]);
          if (j + 1 < n) if (elect_one()) mma_commit(&empty[k.stage]);
        }
      }
      if (elect_one()) mma_commit(mma_done);
      mbar_wait_warp(mma_done, 0, quiet);
    }
  } else if (live && !behind) {
    regs_raise<kAttnFwdRegsHigh>();
    // ---------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2;
    const int row = t.row0 + x * T + (warp & 3) * 32 + lane;
    const int nx = x == 0 ? n_a : (tiles_x == 2 ? n : 0);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + x * T + lanes, tO = tbase + 256 + x * T + lanes;
    const int see = min(max(row + 1, t.prefix_end), t.end);              // keys [begin, see)
    const int all = min(max(t.row0 + x * T + 1, t.prefix_end), t.end);   // ... that every row sees
    const AttnScore<kCap, kBias> score(p, h);
    float m = -INFINITY;
    float2 l = make_float2(0.0f, 0.0f);      // two partial sums
    bool ok = true;
    for (int j = 0; j < nx && ok; ++j) {
      const int j0 = t.begin + j * T;
      ok = mbar_wait(&s_full[x], j & 1, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t v[4][32];
      tmem_ld32(tS, v[0]);
      tmem_ld32(tS + 32, v[1]);
      tmem_ld32(tS + 64, v[2]);
      tmem_ld32(tS + 96, v[3]);
      tmem_wait_ld();
      score.template apply<4, true, false>(v, j0 - row, nullptr);
      if (j0 + T > all) {
        const int lim = see - j0;
#pragma unroll
        for (int c = 0; c < T; ++c)
          if (c >= lim) v[c / 32][c % 32] = 0xff800000u;                  // -infinity
      }
      float top[4] = {m, m, m, m};
#pragma unroll
      for (int e = 0; e < 32; e += 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = max3(top[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
      const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
      if (j == 0) {
        m = mx;
      } else {
        const bool grow = mx > m + score.headroom;
        if (__any_sync(0xffffffffu, grow)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[x], (j - 1) & 1, ctl));
          if (!ok) break;
          tc_fence_after();
          const float a = grow ? ex2((m - mx) * score.mul) : 1.0f;
          l = mul2(l, both(a));
          if (grow) m = mx;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st32(tO + c, o);
          }
        }
      }
      // a row without a finite score so far has no p yet
      const bool none = m == -INFINITY;
      const float2 shift = both(none ? 0.0f : -m * score.mul), mul = both(score.mul);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 y = attn_exp2<kAttnFwdPoly>(fma2(pair_of(&v[c][e]), mul, shift), e / 2);
          sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], y);
          w[e / 2] = pack_bf16x2(y.x, y.y);
        }
        tmem_st16(tS + 16 * c, w);
        // the tensor core begins with the first half of the keys
        if (c == 1) attn_publish(&p_full[2 * x], lane);
      }
      attn_publish(&p_full[2 * x + 1], lane);
      if (none) sum[0] = sum[1] = make_float2(0.0f, 0.0f);
      l = add2(l, add2(sum[0], sum[1]));
    }
    if (ok && nx > 0) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[x], (nx - 1) & 1, ctl));
    if (ok && nx > 0) {
      tc_fence_after();
      const float total = l.x + l.y, inv = 1.0f / total;
      const bool mine = row < t.end;
      __nv_bfloat16* out = p.O + (static_cast<size_t>(row) * p.heads + h) * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
        if (mine) attn_store32(out + c, o, inv);
      }
      // natural logarithm of sum exp z
      if (mine) p.lse[static_cast<size_t>(row) * p.heads + h] = (m * score.mul + log2f(total)) * 0.69314718056f;
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
