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
struct AttnParams {
  AttnPlanView plan;
  const __nv_bfloat16 *Q, *K, *V, *dO;
  const float* slopes;           // [heads] or null
  __nv_bfloat16 *O, *dQ, *dK, *dV;
  float* lse;                    // [M x heads]
  float* stat;                   // backward: [2][heads][M], lse log2(e) and delta
  int M, n_docs, heads, kv_heads;
  float scale, cap;              // cap 0: none
};

__device__ __forceinline__ bool attn_plan_ok(const AttnParams& p) {
  if (p.plan.head[kPlanM] == static_cast<uint32_t>(p.M) && p.plan.head[kPlanDocs] == static_cast<uint32_t>(p.n_docs))
    return true;
  atomicOr(p.plan.head, static_cast<uint32_t>(kStatusBadArgument));
  return false;
}

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

// Scores in the exponent of 2.  Without cap and bias the raw products stay as
// they are and `mul` = scale log2(e) is folded into the exponent; with either
// the values become z log2(e) and mul is 1.
//   tanh(y) = 1 - 2 / (1 + exp(2 y)): right at both ends (0 and infinity in
//   the denominator), absolute error a few 2^-24, so cap tanh is off by less
//   than cap 2^-21 in the exponent.
template <bool kCap, bool kBias>
struct AttnScore {
  float mul;        // of a value in the exponent of 2
  float headroom;   // 8 / mul: how far scores may outgrow the running maximum
  float pre, cap2, slope2;
  __device__ __forceinline__ AttnScore(const AttnParams& p, int h) {
    constexpr bool plain = !kCap && !kBias;
    mul = plain ? p.scale * kLog2e : 1.0f;
    headroom = 8.0f / mul;
    pre = kCap ? 2.0f * kLog2e * p.scale / p.cap : p.scale * kLog2e;
    cap2 = kCap ? p.cap * kLog2e : 0.0f;
    slope2 = kBias ? p.slopes[h] * kLog2e : 0.0f;
  }
  __device__ __forceinline__ float tanh_of(float s) const {
    return fmaf(-2.0f, rcp_approx(1.0f + ex2(s * pre)), 1.0f);
  }
  // z log2(e) of one product; dist = i - j.  *t: the tanh (with a cap)
  __device__ __forceinline__ float one(float s, float dist, float* t) const {
    float z = s;
    if constexpr (kCap) { *t = tanh_of(s); z = cap2 * *t; }
    else if constexpr (kBias) z = s * pre;
    if constexpr (kBias) z = fmaf(-slope2, fabsf(dist), z);
    return z;
  }
  // a row's 128 products; dist0 = i - j of the first
  __device__ __forceinline__ void apply(uint32_t (&v)[4][32], int dist0) const {
    if constexpr (kCap || kBias) {
      const float d0 = static_cast<float>(dist0);
      float t;
#pragma unroll
      for (int c = 0; c < 128; ++c)
        v[c / 32][c % 32] = __float_as_uint(one(__uint_as_float(v[c / 32][c % 32]), d0 - static_cast<float>(c), &t));
    }
  }
};

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

// Waits for the last fill of every ring stage that has one (the aborting
// producer's copies in flight); rp: the stage it would fill next.
__device__ __forceinline__ void attn_drain(uint64_t* full, int stages, RingPos rp) {
  volatile uint32_t never = 0u;
  const AbortCtl quiet{&never, nullptr};
  for (int i = 0; i < stages; ++i) {
    if (i < static_cast<int>(rp.stage)) mbar_wait(&full[i], rp.phase, quiet);
    else if (rp.phase != 0u) mbar_wait(&full[i], rp.phase ^ 1u, quiet);
  }
}

// Rows [first, last) of one head's columns of out [M x heads * D] become zero.  Whole CTA.
template <int D>
__device__ __forceinline__ void attn_zero_rows(__nv_bfloat16* out, int heads, int h, int first, int last) {
  const int n = (last - first) * (D / 8);
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    reinterpret_cast<uint4*>(out + (static_cast<size_t>(first + i / (D / 8)) * heads + h) * D)[i % (D / 8)] =
        make_uint4(0u, 0u, 0u, 0u);
}

// 32 fp32 values times `by` as bf16.
__device__ __forceinline__ void attn_store32(__nv_bfloat16* out, const uint32_t (&v)[32], float by) {
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    uint4 w;
    w.x = pack_bf16x2(__uint_as_float(v[e]) * by, __uint_as_float(v[e + 1]) * by);
    w.y = pack_bf16x2(__uint_as_float(v[e + 2]) * by, __uint_as_float(v[e + 3]) * by);
    w.z = pack_bf16x2(__uint_as_float(v[e + 4]) * by, __uint_as_float(v[e + 5]) * by);
    w.w = pack_bf16x2(__uint_as_float(v[e + 6]) * by, __uint_as_float(v[e + 7]) * by);
    *reinterpret_cast<uint4*>(out + e) = w;
  }
}

}  // namespace lora
