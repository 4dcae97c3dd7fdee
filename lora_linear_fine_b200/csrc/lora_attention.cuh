// lora_attention.cuh — attention over packed documents, forward and backward.
//
//   z_ij = cap tanh(scale q_i.k_j / cap) - slope |i - j|     (no cap: scale q_i.k_j; no slopes: no bias)
//   p_ij = exp(z_ij - lse_i),  lse_i = log sum_j exp z_ij,  o_i = sum_j p_ij v_j
// over the keys j that row i sees: those of its own document with j <= i or
// j before the end of the document's prefix.
//   delta_i = do_i.o_i,  dz_ij = p_ij (do_i.v_j - delta_i)
//   ds_ij = scale dz_ij (1 - tanh^2),  dq_i = sum_j ds_ij k_j,  dk_j = sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
#pragma once

#include "lora_norm_rope.cuh"

namespace lora {

// ---------------------------------------------------------------------------
// the plan: the documents of a batch as lists of tiles
// ---------------------------------------------------------------------------
// A tile is up to kAttnTile (the forward: 2 kAttnTile) rows of one document.
// Tiles start at the document's first row, so a tile never holds rows of two
// documents and whatever a document's rows hold stays out of its neighbours.
// Rows behind the last document come as tiles of their own (prefix_end < 0),
// whose outputs are zero.
constexpr int kAttnTile = 128;

struct AttnTileRef {
  int row0;          // first row
  int begin, end;    // the document's rows
  int prefix_end;    // first row past the document's prefix; -1: rows behind the last document
};

// The plan's header, words of 4 bytes (word 0 is the status word).
enum : int {
  kPlanM = 16,           // rows the plan was made for
  kPlanDocs = 17,
  kPlanFwd = 18,         // tiles in each list
  kPlanQ = 19,
  kPlanKv = 20,
  kPlanCausal = 21,
};

struct AttnPlanView {
  uint32_t* head;
  AttnTileRef* fwd;      // 2 kAttnTile query rows
  AttnTileRef* q;        // kAttnTile query rows
  AttnTileRef* kv;       // kAttnTile key rows
  int max_fwd, max_q;    // capacities (kv: as q)
};

constexpr int kPlanBuckets = 1024;

// Visits the tiles of every list: f(list, work, tile), work in key (list kv:
// query) tiles of kAttnTile.  A warp takes a document, its lanes the tiles.
template <typename F>
__device__ __forceinline__ void plan_tiles(const int* starts, const int* prefix, int M, int n_docs, int causal, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarp = blockDim.x >> 5;
  for (int d = warp; d <= n_docs; d += nwarp) {
    const bool behind = d == n_docs;
    const int a = starts[d], e = behind ? M : starts[d + 1];
    const int len = e - a;
    if (len <= 0) continue;
    const int pre = behind ? -1 : a + (causal ? (prefix != nullptr ? prefix[d] : 0) : len);
    const int tiles = (len + kAttnTile - 1) / kAttnTile;
    for (int t = lane; t < tiles; t += 32) {
      const int r0 = a + t * kAttnTile;
      const AttnTileRef ref{r0, a, e, pre};
      if (behind) {
        if (t % 2 == 0) f(0, 0, ref);
        f(1, 0, ref);
        f(2, 0, ref);
        continue;
      }
      auto keys = [&](int rows) {
        int last = r0 + rows < e ? r0 + rows : e;
        last = last > pre ? last : pre;
        return (last - a + kAttnTile - 1) / kAttnTile;
      };
      if (t % 2 == 0) f(0, keys(2 * kAttnTile), ref);
      f(1, keys(kAttnTile), ref);
      f(2, r0 < pre ? tiles : tiles - t, ref);
    }
  }
}

// One CTA.  Lists the tiles in falling order of their work (a counting sort,
// work above the last bucket together), so that the tiles handed out last are
// short.  Offsets that do not rise from 0 to at most M, or a prefix longer
// than its document, set the status bit and leave the lists empty.
__global__ void __launch_bounds__(1024)
    attn_plan_kernel(const int* __restrict__ starts, const int* __restrict__ prefix, int M, int n_docs, int causal,
                     AttnPlanView v) {
  __shared__ int count[3][kPlanBuckets];
  __shared__ int bad;
  grid_dep_wait();
  if (threadIdx.x == 0) bad = 0;
  for (int i = threadIdx.x; i < 3 * kPlanBuckets; i += blockDim.x) (&count[0][0])[i] = 0;
  __syncthreads();
  bool b = false;
  for (int d = threadIdx.x; d <= n_docs; d += blockDim.x) {
    const int a = starts[d];
    if (a < 0 || a > M || (d == 0 && a != 0)) b = true;
    if (d < n_docs) {
      const int e = starts[d + 1];
      if (e < a || e > M) b = true;
      else if (causal && prefix != nullptr && (prefix[d] < 0 || prefix[d] > e - a)) b = true;
    }
  }
  if (b) bad = 1;
  __syncthreads();
  const bool good = bad == 0;
  if (threadIdx.x == 0) {
    v.head[0] = good ? 0u : static_cast<uint32_t>(kStatusBadArgument);
    v.head[kPlanM] = static_cast<uint32_t>(M);
    v.head[kPlanDocs] = static_cast<uint32_t>(n_docs);
    v.head[kPlanCausal] = static_cast<uint32_t>(causal);
    if (!good) v.head[kPlanFwd] = v.head[kPlanQ] = v.head[kPlanKv] = 0u;
  }
  if (!good) return;
  auto bucket = [](int work) { return kPlanBuckets - 1 - (work < kPlanBuckets ? work : kPlanBuckets - 1); };
  plan_tiles(starts, prefix, M, n_docs, causal,
             [&](int list, int work, const AttnTileRef&) { atomicAdd(&count[list][bucket(work)], 1); });
  __syncthreads();
  // exclusive sums over the buckets, one warp a list
  if (threadIdx.x < 96) {
    const int list = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int run = 0;
    for (int i0 = 0; i0 < kPlanBuckets; i0 += 32) {
      const int c = count[list][i0 + lane];
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      count[list][i0 + lane] = run + s - c;
      run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) v.head[kPlanFwd + list] = static_cast<uint32_t>(run);
  }
  __syncthreads();
  AttnTileRef* lists[3] = {v.fwd, v.q, v.kv};
  plan_tiles(starts, prefix, M, n_docs, causal, [&](int list, int work, const AttnTileRef& ref) {
    lists[list][atomicAdd(&count[list][bucket(work)], 1)] = ref;
  });
}

// ---------------------------------------------------------------------------
// kernels
// ---------------------------------------------------------------------------
// How products become values (AttnScore).
enum AttnTanh { kNoCap, kNearCap, kFarCap };

struct AttnParams {
  AttnPlanView plan;
  const __nv_bfloat16 *Q, *K, *V, *dO;
  const float* slopes;           // [heads] or null
  __nv_bfloat16 *O, *dQ, *dK, *dV;
  float* lse;                    // [M x heads]
  float* stat;                   // backward: [2][heads][M], lse log2(e) and delta
  float* partial;                // backward: [parts][2][M x kv_heads * D] sums of dk and dv (parts > 1)
  int parts, parts_log2;
  int single;                    // forward: items of one tile
  int M, n_docs, causal, heads, kv_heads;
  float scale, cap;              // cap 0: none
  AttnTanh form;
};

__device__ __forceinline__ bool attn_plan_ok(const AttnParams& p) {
  if (p.plan.head[kPlanM] == static_cast<uint32_t>(p.M) && p.plan.head[kPlanDocs] == static_cast<uint32_t>(p.n_docs) &&
      p.plan.head[kPlanCausal] == static_cast<uint32_t>(p.causal))
    return true;
  atomicOr(p.plan.head, static_cast<uint32_t>(kStatusBadArgument));
  return false;
}

// What a persistent CTA works on: (tile, head) pairs, the heads of a tile next
// to each other, tiles in falling order of their work.  The CTAs take them in
// rounds whose direction alternates, so that the sums of their work stay close.
// Each role of a CTA walks over the same items; the next one's tile is loaded
// while it is at the one before.
struct AttnItems {
  AttnTileRef t;
  int h;
  __device__ __forceinline__ AttnItems(const AttnTileRef* list, uint32_t tiles, int heads)
      : t{0, 0, 0, 0}, h(0), list_(list), heads_(static_cast<uint32_t>(heads)), total_(tiles * heads_),
        inverse_(0xffffffffu / heads_) {
    fetch();
  }
  __device__ __forceinline__ bool advance() {
    if (!more_) return false;
    t = next_;
    h = next_h_;
    ++round_;
    fetch();
    return true;
  }
  __device__ __forceinline__ bool behind() const { return t.prefix_end < 0; }

 private:
  __device__ __forceinline__ void fetch() {
    const uint32_t at = round_ * gridDim.x + ((round_ & 1u) ? gridDim.x - 1u - blockIdx.x : blockIdx.x);
    more_ = at < total_;
    if (!more_) return;
    // at / heads: the product with the inverse is the quotient or one less (at < 2^31)
    uint32_t q = __umulhi(at, inverse_), r = at - q * heads_;
    if (r >= heads_) { ++q; r -= heads_; }
    next_h_ = static_cast<int>(r);
    next_ = list_[q];
  }
  const AttnTileRef* list_;
  uint32_t heads_, total_, inverse_, round_ = 0;
  bool more_ = false;
  int next_h_ = 0;
  AttnTileRef next_{0, 0, 0, 0};
};

// Key tiles that the `rows` rows from row0 on see.
__device__ __forceinline__ int attn_key_tiles(const AttnTileRef& t, int row0, int rows) {
  const int see = max(min(row0 + rows, t.end), t.prefix_end);
  return (see - t.begin + kAttnTile - 1) / kAttnTile;
}

// 2^x, the hardware's approximation (relative error below 2^-22).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x, the hardware's approximation (within 1 unit in the last place; 1 / inf = 0).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// The larger of three values (NaN only if all are).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 pair_of(const uint32_t* v) {
  return make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
}

// 2^x of a pair on the FMA pipe: x = n + f with n whole and |f| <= 1/2 (adding
// 1.5 * 2^23 leaves n in the low bits), 2^f by a polynomial of degree 5 that is
// 1 at 0 with the least largest relative error on that interval (2^-22.5 in
// fp32), times 2^n.  From -127 down the result is 0 (the factor's exponent field
// is).  NaN stays NaN, which n added to the bits of p would not leave.  The special function unit gives 16 exponentials a
// cycle and SM, fewer than a tile's products leave time for; so the kernels
// form part of them this way.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  constexpr float kRound = 12582912.0f;
  x = make_float2(max_nan(x.x, -127.0f), max_nan(x.y, -127.0f));
  const float2 t = add2(x, both(kRound));
  const float2 f = fma2(add2(t, both(-kRound)), both(-1.0f), x);
  float2 p = fma2(both(0.001326472731307149f), f, both(0.009671512991189957f));
  p = fma2(p, f, both(0.05550733581185341f));
  p = fma2(p, f, both(0.24022242426872253f));
  p = fma2(p, f, both(0.6931470036506653f));
  p = fma2(p, f, both(1.0f));
  return mul2(p, make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                             __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u)));
}

// 2^x of the i-th pair of a row: kPoly of four pairs by the polynomial.
template <int kPoly>
__device__ __forceinline__ float2 attn_exp2(float2 x, int i) {
  return (i & 3) < kPoly ? exp2_poly(x) : make_float2(ex2(x.x), ex2(x.y));
}

// A score's exponent of 2 is value * mul - slope2 |i - j|.  Without a cap the
// values are the raw products and mul = scale log2(e).  With one they are
// top * tanh(y), y = scale / cap * product, and mul = cap log2(e) / top:
//   tanh(y) = y P(y^2), P of degree 3 with the least largest error for
//   |y| <= 0.4 (2^-23.3): FMAs alone, 5 for a pair where the powers of
//   scale / cap can be folded into P's coefficients.  Else
//   tanh(y) = 1 - 2 / (1 + exp(2 y)), two special functions a value, right at
//   both ends (0 and infinity in the denominator), within a few 2^-24.
//   Each value goes by its own size, so it is the same bits whatever its
//   neighbours in the tile are, which may be another document's; only the work
//   for the second form depends on whether some value of the warp needs it.
// kNearCap (scale / cap within (2^-17, 2^16)): top = 1, scale / cap is folded
// into P.  kFarCap, for the others: y is formed first, since the folded
// coefficients would leave fp32's range; with a cap far above the scores (as
// good as none) top = cap / scale, so that values are near the products and
// nothing is multiplied by the cap (an error of 2^-24 would be one of 2^-24 cap
// in the score), with a cap far below the scale top = 1.  kFarCap is kernels of
// its own: one for both, with its constants among the parameters, took the
// forward 333 us for 291 where scores pass 0.4 of the cap (2 x 4096 tokens, 16 /
// 4 heads of 128, cap 30).
template <AttnTanh kTanh, bool kBias>
struct AttnScore {
  static constexpr bool kCap = kTanh != kNoCap, kFar = kTanh == kFarCap;
  // Of four pairs of exponentials, those by the polynomial.  With a cap or a
  // bias the FMA pipe is the busy one already.
  static constexpr int kPoly = kCap || kBias ? 0 : 1;
  float mul;
  float slope2 = 0.0f;
  float limit = 0.0f, twice = 0.0f, a0 = 0.0f, a1 = 0.0f, a2 = 0.0f, a3 = 0.0f;
  float turn = 1.0f, top = 1.0f, fall = -1.0f;
  __device__ __forceinline__ explicit AttnScore(const AttnParams& p) : mul((kCap ? p.cap : p.scale) * kLog2e) {
    if constexpr (kCap) {
      float pre = p.scale / p.cap;
      if constexpr (kFar) {
        turn = fminf(pre, 0x1.fffffep127f);
        if (pre < 1.0f) {
          top = p.cap / p.scale;
          mul = p.scale * kLog2e;
        }
        fall = -1.0f / (top * top);
        pre = 1.0f;
      }
      const float u = pre * pre;
      limit = 0.4f / pre;
      twice = 2.0f * kLog2e * pre;
      a0 = 0.9999998807907104f * pre * top;
      a1 = -0.333313912153244f * pre * u * top;
      a2 = 0.1327143758535385f * pre * u * u * top;
      a3 = -0.04757281020283699f * pre * u * u * u * top;
    }
  }
  __device__ __forceinline__ void head(const AttnParams& p, int h) {
    if constexpr (kBias) slope2 = p.slopes[h] * kLog2e;
  }
  // n products of a row become values; dt: 1 - tanh^2 (only with a cap).
  template <bool kWantDt, int n>
  __device__ __forceinline__ void values(uint32_t (&v)[n], float2* dt) const {
    if constexpr (kCap) {
      if constexpr (kFar) {
#pragma unroll
        for (int e = 0; e < n; e += 2) put(v, e, mul2(pair_of(&v[e]), both(turn)));
      }
      float size[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < n; e += 4) {
        size[0] = max3_abs(size[0], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        size[1] = max3_abs(size[1], __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
      }
      if (!__any_sync(0xffffffffu, fmaxf(size[0], size[1]) > limit)) {
#pragma unroll
        for (int e = 0; e < n; e += 2) put(v, e, near(pair_of(&v[e])));
      } else {
#pragma unroll
        for (int e = 0; e < n; e += 2) {
          const float2 s = pair_of(&v[e]), z = near(s);
          put(v, e, make_float2(fabsf(s.x) <= limit ? z.x : far(s.x), fabsf(s.y) <= limit ? z.y : far(s.y)));
        }
      }
      if constexpr (kWantDt) {
#pragma unroll
        for (int e = 0; e < n; e += 2) {
          const float2 t = pair_of(&v[e]);
          dt[e / 2] = fma2(mul2(t, t), both(fall), both(1.0f));
        }
      }
    }
  }
  // one product's value
  __device__ __forceinline__ float one(float s) const {
    if constexpr (!kCap) return s;
    if constexpr (kFar) s *= turn;
    return fabsf(s) <= limit ? near(both(s)).x : far(s);
  }
  __device__ __forceinline__ float2 near(float2 s) const {
    const float2 u = mul2(s, s);
    float2 q = fma2(both(a3), u, both(a2));
    q = fma2(q, u, both(a1));
    q = fma2(q, u, both(a0));
    return mul2(s, q);
  }
  __device__ __forceinline__ float far(float s) const {
    return fmaf(-2.0f * top, rcp_approx(1.0f + ex2(s * twice)), top);
  }
  // `base` minus the bias at distances d0 + c and d0 + c + 1 (either sign)
  __device__ __forceinline__ float2 shifted(float2 base, float d0, float c, float step) const {
    if constexpr (!kBias) return base;
    const float2 d = add2(both(d0), make_float2(c, c + step));
    return make_float2(fmaf(-slope2, fabsf(d.x), base.x), fmaf(-slope2, fabsf(d.y), base.y));
  }
  template <int n>
  __device__ __forceinline__ static void put(uint32_t (&v)[n], int e, float2 z) {
    v[e] = __float_as_uint(z.x);
    v[e + 1] = __float_as_uint(z.y);
  }
};

constexpr float kAttnHeadroom = 16.0f;   // exponents of 2 by which scores may outgrow the running reference

// The warp's stores to tensor memory are done: tell the MMA warp.
__device__ __forceinline__ void attn_publish(uint64_t* bar, int lane) {
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A tile of 128 rows x 128 scores is worked on by 128 threads a group of kCols
// columns; each group writes its bf16 results over the first half of its own
// columns, in two parts.  Part c of all groups is four of the eight steps of 16
// that the product over them takes: k = 0 .. 3 -> step, step -> column.
template <int kCols>
__device__ __forceinline__ int attn_part_step(int c, int k) {
  constexpr int n = kCols / 32;          // steps of a part in a group
  return (k / n) * 2 * n + n * c + k % n;
}
template <int kCols>
__device__ __forceinline__ uint32_t attn_step_column(int kk) {
  constexpr int n = kCols / 16;
  return (kk / n) * kCols + 8 * (kk % n);
}

// Zeroes rows [first, kAttnTile) of a tile of kBoxes 128-byte column boxes in
// shared memory and makes that visible to the tensor core.  One warp.
template <int kBoxes>
__device__ __forceinline__ void attn_trim_tile(uint8_t* tile, int first, int lane) {
  for (int b = 0; b < kBoxes; ++b) {
    uint4* rows = reinterpret_cast<uint4*>(tile + b * (kAttnTile * 128));
    for (int i = first * 8 + lane; i < kAttnTile * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Waits for the last fill of every ring stage (the aborting producer's copies
// in flight); rp: the stage it would fill next.  A stage without a fill passes.
__device__ __forceinline__ void attn_drain(uint64_t* full, int stages, RingPos rp) {
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};
  for (int i = 0; i < stages; ++i)
    mbar_wait(&full[i], i < static_cast<int>(rp.stage) ? rp.phase : rp.phase ^ 1u, quiet);
}

// Rows [first, last) of one head's columns of out [M x heads * D] become zero.
// Thread i of n.
template <int D>
__device__ __forceinline__ void attn_zero_rows(__nv_bfloat16* out, int heads, int h, int first, int last, int i, int n) {
  for (; i < (last - first) * (D / 8); i += n)
    reinterpret_cast<uint4*>(out + (static_cast<size_t>(first + i / (D / 8)) * heads + h) * D)[i % (D / 8)] =
        make_uint4(0u, 0u, 0u, 0u);
}

// fp32 values times `by` as bf16.
__device__ __forceinline__ uint4 attn_pack8(const uint32_t* v, float by) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = mul2(pair_of(v + 2 * k), both(by));
    w[k] = pack_bf16x2(y.x, y.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Each lane holds n 16-byte chunks of its own row (lane i: row i of the warp's
// 32): they change places within groups of n lanes, so that a store writes
// whole 16 n byte pieces of 32 / n rows.  32 rows at a time, one chunk each,
// cost the store path a cycle or two a row: 3700 cycles for a tile of dk and
// dv.  Rows from `rows` on are left out.
template <int n>
__device__ __forceinline__ void attn_store_rows(uint4 (&w)[n], uint8_t* base, size_t stride, int rows, int lane) {
#pragma unroll
  for (int s = n / 2; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if (i & s) continue;
      uint4 v = up ? w[i] : w[i | s];
      v.x = __shfl_xor_sync(0xffffffffu, v.x, s);
      v.y = __shfl_xor_sync(0xffffffffu, v.y, s);
      v.z = __shfl_xor_sync(0xffffffffu, v.z, s);
      v.w = __shfl_xor_sync(0xffffffffu, v.w, s);
      if (up) w[i] = v;
      else w[i | s] = v;
    }
  }
  const int first = lane / n * n;
  uint8_t* out = base + first * stride + (lane % n) * 16;
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (first + i < rows) *reinterpret_cast<uint4*>(out + i * stride) = w[i];
}

}  // namespace lora
