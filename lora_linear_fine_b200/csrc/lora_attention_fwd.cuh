// lora_attention_fwd.cuh — the attention forward on the tensor cores.
//
// A persistent CTA (one an SM) works through items of up to 256 query rows of
// one document and one head: two tiles of 128 rows, a and b, that share the
// key / value tiles of 128 rows.  For each key tile j, the nearest first, and
// each of a, b:
//   S = Q K_j^T          tcgen05.mma, both operands in shared memory, S in tensor memory
//   P = exp2(z - m)      a warpgroup, one thread a row: S to registers, bf16 P back over S
//   O += P V_j           tcgen05.mma with P read from tensor memory
// so the scores never leave the SM.  While one warpgroup works on its S the
// tensor core works for the other one, and the next item's loads and first
// products run under this one's last softmax and stores.  Tensor memory: S a,
// S b (128 columns each, P over their first 64), O a, O b.
//
// One warp issues the products of both, so that they alternate: with a warp
// each, both tiles fall into step, and the tensor core idles while both are at
// their softmax (measured: 10% slower).
//
// m is a reference, not the maximum itself: it starts as the maximum of the
// row's first tile and moves only when a later score lies more than 2^16 above
// it.  Until then P and the row's sum l are larger by the same factor, which
// fp32 and bf16 hold as well, and the rescaling of O in tensor memory (a read
// and a write of all of it) is rare.  Scores under a cap up to 55 need no
// maximum: exponents of 2 within +-80 are taken as they are (m = 0; V may lie
// within 2^+-26 over rows of 2^20 keys even where all scores are at the cap).
// P is rounded to bf16 for the tensor core; l adds the fp32 values.
//
// The softmax goes through its 128 columns in pieces of 32, in loops that are
// not unrolled: all of it in registers and in line is 40 KB of code with a cap
// and a bias, and its two warpgroups then wait for instructions.
#pragma once

#include "lora_attention.cuh"

namespace lora {

template <int D>
struct AttnFwdCfg {
  static constexpr int kBoxes = D / 64;                          // 128-byte column boxes of a tile
  static constexpr int kTileBytes = kAttnTile * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;               // K and V tiles in flight
  static constexpr int kBars = 3 * kStages + 2 + 2 + 4 + 2 + 2 + 1;
  static constexpr int kSmemBytes = (2 + kStages) * kTileBytes + kBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= kSmemLimitBytes, "shared memory");
};
constexpr int kAttnFwdThreads = 384;     // warps: TMA, MMA, trimming, one idle, softmax of tile a (4), of tile b (4)

constexpr float kAttnFixedRange = 80.0f;

struct AttnFwdMaps {
  CUtensorMap q, k, v;     // [M x heads * D] bf16, box 64 x 128, 128-byte swizzle
};

template <int D, AttnTanh kTanh, bool kBias>
__global__ void __launch_bounds__(kAttnFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnFwdMaps maps) {
  using C = AttnFwdCfg<D>;
  constexpr bool kCap = kTanh != kNoCap;
  constexpr int T = kAttnTile, S = C::kStages, kPoly = AttnScore<kTanh, kBias>::kPoly;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * C::kTileBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * C::kTileBytes);
  uint64_t* empty = full + S;
  uint64_t* land = empty + S;        // [S] a tile that is trimmed before it counts as full
  uint64_t* q_full = land + S;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;    // [2] S of this key tile is in tensor memory
  uint64_t* p_full = s_full + 2;     // [2][2] that half of P is in tensor memory (and O rescaled)
  uint64_t* pv_done = p_full + 4;    // [2] O holds this key tile
  uint64_t* o_empty = pv_done + 2;   // [2] O has been read
  uint64_t* mma_done = o_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  AbortCtl ctl{abort_flag, p.plan.head};
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); mbar_init(&land[i], 1); }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&o_empty[x], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // Tensor memory is held before a dependent kernel may start (grid_dep_wait),
  // so none of its CTAs can take what a CTA of this grid still waits for.
  grid_dep_wait();

  // Items of one tile where pairs would leave SMs idle.
  AttnItems items(p.single ? p.plan.q : p.plan.fwd, attn_plan_ok(p) ? p.plan.head[p.single ? kPlanQ : kPlanFwd] : 0u,
                  p.heads);
  auto pair = [&] { return !p.single && items.t.row0 + T < items.t.end; };
  bool ok = true;
  // key tiles that the rows of the item's two tiles see
  auto tiles_of = [&](int* n_a) {
    *n_a = attn_key_tiles(items.t, items.t.row0, T);
    return pair() ? attn_key_tiles(items.t, items.t.row0 + T, T) : *n_a;
  };

  if (warp < 4) {
    if (warp == 0) {
      // -------------------------------------------------------------- TMA
      if (lane == 0) {
        RingPos rp;
        uint32_t q_turn = 0;
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const AttnTileRef t = items.t;
          const int h = items.h, hk = h / (p.heads / p.kv_heads);
          const int tiles_x = pair() ? 2 : 1;
          int n_a;
          const int n = tiles_of(&n_a);
          for (int i = 0; i < 2 * n && ok; ++i) {
            const bool is_v = i & 1;
            const int row = t.begin + (n - 1 - i / 2) * T;
            ok = mbar_wait(&empty[rp.stage], rp.phase ^ 1u, ctl);
            if (!ok) break;
            // Rows past the document in its last value tile are zeroed: their
            // P is zero, but zero times an infinity or NaN there would not be.
            uint64_t* bar = is_v && row + T > t.end ? &land[rp.stage] : &full[rp.stage];
            uint8_t* dst = ring + rp.stage * C::kTileBytes;
            mbar_arrive_expect_tx(bar, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_2d(dst + b * (T * 128), is_v ? &maps.v : &maps.k, bar, hk * D + 64 * b, row);
            rp.next(S);
            if (i == 0) {
              ok = mbar_wait(q_empty, (q_turn & 1u) ^ 1u, ctl);
              if (!ok) break;
              ++q_turn;
              mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tiles_x * C::kTileBytes));
              for (int x = 0; x < tiles_x; ++x)
                for (int b = 0; b < C::kBoxes; ++b)
                  tma_load_2d(smem + x * C::kTileBytes + b * (T * 128), &maps.q, q_full, h * D + 64 * b, t.row0 + x * T);
            }
          }
        }
        if (!ok) {   // every copy has landed before the CTA may end
          mbar_wait(q_full, (q_turn & 1u) ^ 1u, quiet);
          attn_drain(full, S, rp);
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA
      if (elect_one()) {
        constexpr uint32_t kIdS = idesc_bf16(T, T, false, false);
        constexpr uint32_t kIdO = idesc_bf16(T, D, false, true);
        const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t k_desc = sdesc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t v_desc = sdesc_sw128(smem_u32(ring), T * 128, 1024);
        auto scores = [&](int x, uint32_t stage) {
          const uint64_t a = q_desc + x * (C::kTileBytes >> 4), b = k_desc + stage * (C::kTileBytes >> 4);
          {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * (T * 128) + (kk % 4) * 32) >> 4;
              mma_bf16(tbase + x * T, a + off, b + off, kIdS, kk > 0);
            }
            mma_commit(&s_full[x]);
          }
        };
        // half of the keys: 4 steps of 16
        auto values = [&](int x, uint32_t stage, int half, bool first) {
          const uint64_t b = v_desc + stage * (C::kTileBytes >> 4);
          {
#pragma unroll
            for (int k = 0; k < T / 32; ++k) {
              const int kk = half * (T / 32) + k;
              mma_bf16_ta(tbase + 256 + x * T, tbase + x * T + 8 * kk, b + kk * (2048 >> 4), kIdO, !first || kk > 0);
            }
            if (half == 1) mma_commit(&pv_done[x]);
          }
        };
        RingPos rp;
        uint32_t q_turn = 0, o_turn[2] = {0, 0}, step[2] = {0, 0};      // of Q; of O; key tiles of a and b
        while (ok && items.advance()) {
          if (items.behind()) continue;
          const int tiles_x = pair() ? 2 : 1;
          int n_a;
          const int n = tiles_of(&n_a);
          // tile a begins with its own first key tile, which may be b's second
          const int skip = n - n_a;
          ok = mbar_wait(q_full, q_turn & 1u, ctl) && mbar_wait(&full[rp.stage], rp.phase, ctl);
          if (!ok) break;
          ++q_turn;
          tc_fence_after();
          RingPos v = rp;
          v.next(S);
          RingPos k = v;
          k.next(S);
          if (skip == 0) scores(0, rp.stage);
          if (tiles_x == 2) scores(1, rp.stage);
          mma_commit(&empty[rp.stage]);
          if (n == 1) mma_commit(q_empty);
          ok = mbar_wait(&full[v.stage], v.phase, ctl);
          if (n > 1) ok = ok && mbar_wait(&full[k.stage], k.phase, ctl);
          tc_fence_after();
          for (int j = 0; j < n && ok; ++j) {
            // the next turn's tiles, waited for while there is time
            RingPos v2 = k, k2 = k;
            v2.next(S);
            k2.next(S);
            k2.next(S);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int from = x == 0 ? skip : 0;
              if (ok && j >= from && x < tiles_x) {
                if (j == from) ok = mbar_wait(&o_empty[x], (o_turn[x]++ & 1u) ^ 1u, ctl);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  ok = ok && mbar_wait(&p_full[2 * x + half], step[x] & 1u, ctl);
                  if (!ok) break;
                  tc_fence_after();
                  values(x, v.stage, half, j == from);
                }
                ++step[x];
              }
              if (ok && j + 1 >= from && j + 1 < n && x < tiles_x) scores(x, k.stage);
              if (x == 0 && ok && j + 1 < n) {
                ok = mbar_wait(&full[v2.stage], v2.phase, ctl);
                if (j + 2 < n) ok = ok && mbar_wait(&full[k2.stage], k2.phase, ctl);
                tc_fence_after();
              }
            }
            if (ok) {
              mma_commit(&empty[v.stage]);
              if (j + 1 < n) mma_commit(&empty[k.stage]);
              if (j + 2 == n) mma_commit(q_empty);        // the last scores have been issued
            }
            rp = k;
            v = v2;
            k = k2;
          }
        }
        mma_commit(mma_done);
        mbar_wait(mma_done, 0, quiet);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- trimming
      uint32_t slot = 0, landed = 0;         // ring slots so far; a bit a stage: parity of its next landing
      while (ok && items.advance()) {
        if (items.behind()) continue;
        int n_a;
        const int n = tiles_of(&n_a);
        const int row = items.t.begin + (n - 1) * T;
        if (row + T > items.t.end) {           // the first value tile of the item
          const uint32_t stage = (slot + 1) % S;
          ok = mbar_wait_warp(&land[stage], (landed >> stage) & 1u, ctl);
          if (!ok) break;
          landed ^= 1u << stage;
          attn_trim_tile<C::kBoxes>(ring + stage * C::kTileBytes, items.t.end - row, lane);
          if (lane == 0) mbar_arrive(&full[stage]);
        }
        slot += 2 * n;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + x * T + lanes, tO = tbase + 256 + x * T + lanes;
    AttnScore<kTanh, kBias> score(p);
    const float2 mul = both(score.mul);
    uint32_t step = 0;                       // key tiles of this warpgroup so far
    while (ok && items.advance()) {
      const AttnTileRef t = items.t;
      const int h = items.h;
      if (items.behind()) {
        const int last = min(t.row0 + (p.single ? T : 2 * T), t.end);
        attn_zero_rows<D>(p.O, p.heads, h, t.row0, last, threadIdx.x - 128, 256);
        const int r = t.row0 + static_cast<int>(threadIdx.x) - 128;
        if (r < last) p.lse[static_cast<size_t>(r) * p.heads + h] = -INFINITY;
        continue;
      }
      const int row = t.row0 + x * T + (warp & 3) * 32 + lane;
      const bool mine = row < t.end;         // rows past the document decide nothing
      int n_a;
      const int n = tiles_of(&n_a);
      const int nx = x == 0 ? n_a : (pair() ? n : 0);
      const int see = min(max(row + 1, t.prefix_end), t.end);              // keys [begin, see)
      const int all = min(max(t.row0 + x * T + 1, t.prefix_end), t.end);   // ... that every row sees
      score.head(p, h);
      // rows of few keys take their maximum: p of the only key, or of one that
      // outweighs the others, is then 1 and needs no rounding
      const bool fixed = kCap && nx > 1 && p.cap * kLog2e <= kAttnFixedRange && score.slope2 >= 0.0f;
      float m = fixed ? 0.0f : -INFINITY;      // the reference, an exponent of 2
      float2 l = make_float2(0.0f, 0.0f);      // two partial sums
      for (int j = nx - 1; j >= 0 && ok; --j, ++step) {
        const int j0 = t.begin + j * T;
        const float d0 = static_cast<float>(j0 - row);
        const bool part = j0 + T > all;
        ok = mbar_wait_warp(&s_full[x], step & 1u, ctl);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[2][32];
        auto fetch = [&](int half) {
          tmem_ld32(tS + 64 * half, v[0]);
          tmem_ld32(tS + 64 * half + 32, v[1]);
        };
        auto hide = [&](int half) {
          const int lim = see - j0 - 64 * half;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= lim) v[c / 32][c % 32] = 0xff800000u;                // -infinity
        };
        // The largest exponent of the row in this tile: exact, or with a bias
        // from the largest value and the largest bias apart.
        auto largest = [&](bool exact) {
          float u[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            fetch(half);
            tmem_wait_ld();
            if (kBias && exact) {
              score.template values<false>(v[0], nullptr);
              score.template values<false>(v[1], nullptr);
            }
            if (part) hide(half);        // after the cap, which would make a score of the mask
            if (kBias && exact) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float2 z = fma2(pair_of(&v[c][e]), mul, score.shifted(both(0.0f), d0 + 64 * half, 32 * c + e, 1.0f));
                  u[c] = max3(u[c], z.x, z.y);
                }
            } else {
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                  u[c] = max3(u[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
            }
          }
          const float top = fmaxf(u[0], u[1]);
          if (kBias && exact) return top;
          const float z = score.one(top) * score.mul;
          if constexpr (!kBias) return z;
          const float far = fmaxf(fabsf(d0), fabsf(d0 + (T - 1))), near = max3(0.0f, d0, -d0 - (T - 1));
          return z + fmaxf(-score.slope2 * far, -score.slope2 * near);
        };
        if (!fixed) {
          // a row without a finite score so far has neither a reference nor any sums
          const bool fresh = __any_sync(0xffffffffu, mine && m == -INFINITY);
          float mx = largest(fresh);
          if (fresh && m == -INFINITY) m = mx;
          bool grow = mine && mx > m + kAttnHeadroom;
          if (__any_sync(0xffffffffu, grow)) {
            if (kBias && !fresh) {
              mx = largest(true);
              grow = mine && mx > m + kAttnHeadroom;
            }
            if (j < nx - 1 && __any_sync(0xffffffffu, grow)) {
              ok = mbar_wait_warp(&pv_done[x], (step - 1) & 1u, ctl);
              if (!ok) break;
              tc_fence_after();
              const float a = grow ? ex2(m - mx) : 1.0f;
              l = mul2(l, both(a));
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                tmem_st32(tO + c, o);
              }
            }
            if (grow) m = mx;
          }
        }
        const bool none = m == -INFINITY;
        const float2 shift = both(none ? 0.0f : -m);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        fetch(0);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          tmem_wait_ld();
          score.template values<false>(v[0], nullptr);
          score.template values<false>(v[1], nullptr);
          if (part) hide(half);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = attn_exp2<kPoly>(
                  fma2(pair_of(&v[c][e]), mul, score.shifted(shift, d0 + 64 * half, 32 * c + e, 1.0f)), e / 2);
              sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], y);
              w[e / 2] = pack_bf16x2(y.x, y.y);
            }
            tmem_st16(tS + 32 * half + 16 * c, w);
          }
          if (half == 0) fetch(1);
          attn_publish(&p_full[2 * x + half], lane);       // the tensor core begins with the first half of the keys
        }
        l = add2(l, add2(sum[0], sum[1]));
      }
      if (!ok || nx == 0) continue;
      ok = mbar_wait_warp(&pv_done[x], (step - 1) & 1u, ctl);
      if (!ok) break;
      tc_fence_after();
      const float total = l.x + l.y, inv = 1.0f / total;
      const int row0 = row - lane;               // the warp's first
      const size_t stride = static_cast<size_t>(p.heads) * D * 2;
      uint8_t* out = reinterpret_cast<uint8_t*>(p.O) + row0 * stride + static_cast<size_t>(h) * D * 2;
#pragma unroll
      for (int f = 0; f < D; f += 64) {
        uint4 w[8];
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + f + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 8) w[(c + e) / 8] = attn_pack8(&o[e], inv);
        }
        if (f + 64 == D) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[x]);
        }
        attn_store_rows<8>(w, out + f * 2, stride, t.end - row0, lane);
      }
      if (mine) {
        // natural logarithm of sum exp z
        p.lse[static_cast<size_t>(row) * p.heads + h] = (m + log2f(total)) * 0.69314718056f;
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
