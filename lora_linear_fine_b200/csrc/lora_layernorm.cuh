// lora_layernorm.cuh — layer norm with trained scale and shift, forward and
// backward, beside the RMSNorm prologue (lora_norm_rope.cuh).
//
//   mean = sum_j x_j / d,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / d + eps)
//   xh = (x - mean) rstd,  y = xh g + b                           (per token)
//   dh = dy g,  dx = rstd (dh - mean_j(dh) - xh mean_j(dh xh))
//   dg = sum_m dy xh,  db = sum_m dy
//
// Both directions are bound by memory, so what counts is that loads are always
// in flight.  The forward keeps a row in the registers of a group of T threads
// (16 features a thread) and has loaded the next row before it reduces this
// one.  The backward streams blocks of rows into a ring in shared memory by
// bulk copies (up to 200 KB in flight an SM; the registers hold dg and db of
// the columns instead) and writes one partial row of dg and db a CTA, which
// layernorm_reduce_kernel adds in a fixed order: the same bits in every call.
#pragma once

#include "lora_norm_rope.cuh"

namespace lora {

constexpr int kLnMaxD = 16384;       // 1024 threads x 16 features
constexpr int kLnNV = 2;             // 16-byte chunks a thread
constexpr int kLnSums = 4;           // most sums taken at once

template <int T>
struct LnCfg {
  static constexpr int kThreads = T > 256 ? T : 256;
  static constexpr int kGroups = kThreads / T;     // rows a CTA works on at a time
  static constexpr int kWarps = T / 32;            // warps a row
  static constexpr int kPerSm = T > 512 ? 1 : T > 256 ? 2 : T == 256 ? 5 : 4;     // CTAs an SM of the forward
};

// Sums of `n` values over the T threads of a group, the same in every thread:
// a butterfly within the warps, the warps' sums through `slots` (one row of
// kWarps x kLnSums floats a group, alternating between two rows so that one barrier
// a call is enough).
template <int T, int n, int kGroups = LnCfg<T>::kGroups>
__device__ __forceinline__ void ln_group_sum(float (&v)[n], float* slots, int group, uint32_t& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    const int w = (threadIdx.x % T) >> 5, lane = threadIdx.x & 31;
    float* s = slots + ((phase & 1u) * kGroups + group) * (W * kLnSums);
    ++phase;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < n; ++i) s[w * n + i] = v[i];
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = lane < W ? s[lane * n + i] : 0.0f;
#pragma unroll
    for (int o = (W > 16 ? 16 : W / 2); o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
  }
}

__device__ __forceinline__ void ln_unpack8(uint4 w, float2 (&f)[4]) {
  f[0] = unpack_bf16x2(w.x); f[1] = unpack_bf16x2(w.y); f[2] = unpack_bf16x2(w.z); f[3] = unpack_bf16x2(w.w);
}

// CTAs an SM: as many as the registers of a row in hand and the next one allow.
// 1 / d comes as the sum of two fp32 numbers, so that the mean is rounded once: a
// row of one value has exactly that mean, and x - mean is zero.  With 1 / d
// rounded to one the mean could be a step off, which 1 / sqrt(eps) multiplies.
// (16384 x 4096: 47.2 us, with a rounded 1 / d 46.8, with a division 47.8.)
template <int T>
__global__ void __launch_bounds__(LnCfg<T>::kThreads, LnCfg<T>::kPerSm)
    layernorm_fwd_kernel(const __nv_bfloat16* X, const __nv_bfloat16* __restrict__ g,
                         const __nv_bfloat16* __restrict__ b, long long M, int d, float inv_d, float inv_d_rest,
                         float eps, __nv_bfloat16* Y, float* __restrict__ mean, float* __restrict__ rstd) {
  using C = LnCfg<T>;
  __shared__ float slots[2 * C::kGroups * C::kWarps * kLnSums];
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  const int nv = d / 8;
  uint32_t phase = 0;
  grid_dep_wait();
  const long long step = static_cast<long long>(gridDim.x) * C::kGroups;
  long long row = blockIdx.x * static_cast<long long>(C::kGroups) + group;
  uint4 next[kLnNV];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      next[v] = r < M && c < nv ? reinterpret_cast<const uint4*>(X + r * d)[c] : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(row);
  for (; row < M; row += step) {
    float2 x[kLnNV][4], two = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      ln_unpack8(next[v], x[v]);
#pragma unroll
      for (int e = 0; e < 4; ++e) two = add2(two, x[v][e]);
    }
    fetch(row + step);
    float s[1] = {two.x + two.y};
    ln_group_sum<T, 1>(s, slots, group, phase);
    const float mu = fmaf(s[0], inv_d, s[0] * inv_d_rest);
    two = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int v = 0; v < kLnNV; ++v)
      if (t + v * T < nv)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 dx = add2(x[v][e], both(-mu));
          two = fma2(dx, dx, two);
        }
    s[0] = two.x + two.y;
    ln_group_sum<T, 1>(s, slots, group, phase);
    const float rs = 1.0f / sqrtf(s[0] * inv_d + eps);
    if (t == 0) {
      mean[row] = mu;
      rstd[row] = rs;
    }
    uint4* yr = reinterpret_cast<uint4*>(Y + row * d);
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      if (c >= nv) break;
      float2 w[4], sh[4];
      ln_unpack8(__ldg(reinterpret_cast<const uint4*>(g) + c), w);
      ln_unpack8(b != nullptr ? __ldg(reinterpret_cast<const uint4*>(b) + c) : make_uint4(0u, 0u, 0u, 0u), sh);
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = fma2(mul2(add2(x[v][e], both(-mu)), both(rs)), w[e], sh[e]);
        y[e] = pack_bf16x2(u.x, u.y);
      }
      yr[c] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

__device__ __forceinline__ void ln_load8(const __nv_bfloat16* p, float2 (&f)[4]) {
  ln_unpack8(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void ln_load8(const float* p, float2 (&f)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}

// Layout of the backward: T threads a row, NV chunks of 8 features a thread
// (four for rows wider than 8192: dg and db take half of a thread's 128
// registers then), blocks of rows a ring stage.  Thread 0 issues the copies: a
// warp of its own for that would leave 96 registers a thread, and what then
// goes to local memory misses the little L1 that the ring leaves.
constexpr int kLnBwdThreads = 512;
constexpr int kLnRingBytes = 192 * 1024, kLnStageBytes = 32 * 1024, kLnMaxStages = 8;

struct LnBwdShape {
  int rows;        // rows of a stage
  int stages;
};

// part [gridDim.x][2][d] fp32: each CTA's dg and db over its rows (null: neither is wanted).
template <int T, int NV, typename TDy>
__global__ void __launch_bounds__(kLnBwdThreads, 1)
    layernorm_bwd_kernel(const TDy* dY, const __nv_bfloat16* X, const __nv_bfloat16* __restrict__ g,
                         const float* __restrict__ mean, const float* __restrict__ rstd, long long M, int d,
                         __nv_bfloat16* dX, float* __restrict__ part, LnBwdShape sh, int want_db, uint32_t* status) {
  constexpr int kGroups = kLnBwdThreads / T, kWarps = T / 32;
  constexpr int kQ = NV == 2 ? 2 : 1;      // rows a group takes at a time (a stage of wide rows holds one)
  extern __shared__ __align__(128) uint8_t ln_smem[];          // ring: rows of X, then rows of dY, a stage
  __shared__ float slots[2 * kGroups * kWarps * kLnSums];
  __shared__ uint64_t full[kLnMaxStages], empty[kLnMaxStages];
  __shared__ uint32_t abort_word;
  AbortCtl ctl{&abort_word, status};
  if (threadIdx.x == 0) {
    for (int i = 0; i < sh.stages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], kLnBwdThreads / 32); }
    abort_word = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  const size_t x_bytes = static_cast<size_t>(d) * 2, y_bytes = static_cast<size_t>(d) * sizeof(TDy);
  const size_t stage_bytes = sh.rows * (x_bytes + y_bytes);
  const long long blocks = (M + sh.rows - 1) / sh.rows;
  long long filled = 0, at = 0;          // blocks copied so far, blocks begun
  // Thread 0: block number k of this CTA to its stage, once the block there before has been read.
  auto fill = [&](long long k) {
    const long long blk = blockIdx.x + k * gridDim.x;
    const uint32_t stage = static_cast<uint32_t>(k % sh.stages);
    if (blk >= blocks) return;
    if (k >= sh.stages && !mbar_wait(&empty[stage], static_cast<uint32_t>(k / sh.stages - 1) & 1u, ctl)) return;
    const long long row = blk * sh.rows;
    const long long n = M - row < sh.rows ? M - row : sh.rows;
    uint8_t* dst = ln_smem + stage * stage_bytes;
    const uint32_t xb = static_cast<uint32_t>(n * x_bytes), yb = static_cast<uint32_t>(n * y_bytes);
    mbar_arrive_expect_tx(&full[stage], xb + yb);
    bulk_load_1d(dst, X + row * d, xb, &full[stage]);
    bulk_load_1d(dst + sh.rows * x_bytes, dY + row * d, yb, &full[stage]);
    filled = k + 1;
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < sh.stages; ++k) fill(k);
  // -------------------------------------------------------------------- rows
  const int group = threadIdx.x / T, t = threadIdx.x % T, lane = threadIdx.x & 31;
  const int nv = d / 8;
  const float inv_d = 1.0f / static_cast<float>(d);
  uint32_t phase = 0;
  float2 ag[NV][4], ab[NV][4];
  // g lies in shared memory behind the ring; a thread reads back what it wrote
  __nv_bfloat16* gs = reinterpret_cast<__nv_bfloat16*>(ln_smem + sh.stages * stage_bytes) + group * d;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) ag[v][e] = ab[v][e] = make_float2(0.0f, 0.0f);
    if (t + v * T < nv) reinterpret_cast<uint4*>(gs)[t + v * T] = __ldg(reinterpret_cast<const uint4*>(g) + t + v * T);
  }
  // mean and rstd of the group's next rows, loaded while it is at the ones before
  float mu[kQ], rs[kQ];
  auto stats = [&](long long row0, int k) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const long long row = row0 + k + q * kGroups;
      const bool in = k + q * kGroups < sh.rows && row < M;
      mu[q] = in ? __ldg(mean + row) : 0.0f;
      rs[q] = in ? __ldg(rstd + row) : 0.0f;
    }
  };
  RingPos r;
  bool ok = true;
  stats(blockIdx.x * static_cast<long long>(sh.rows), group);
  for (long long blk = blockIdx.x; blk < blocks && ok; blk += gridDim.x) {
    const long long row0 = blk * sh.rows;
    const int n = static_cast<int>(M - row0 < sh.rows ? M - row0 : sh.rows);
    ok = __all_sync(0xffffffffu, mbar_wait(&full[r.stage], r.phase, ctl));
    if constexpr (T > 32) ok = bar_sync_and<T>(group + 1, ok);          // a group leaves the loop together
    if (!ok) break;
    if (threadIdx.x == 0 && at > 0) fill(at - 1 + sh.stages);
    ++at;
    const uint8_t* xs = ln_smem + r.stage * stage_bytes;
    const uint8_t* ys = xs + sh.rows * x_bytes;
    // kQ rows at a time, so that one round of sums serves them all.  x_hat is
    // (x - mean) rstd, as in the forward: x rstd - mean rstd is an instruction
    // less, but rounds mean rstd, which may be far larger than x_hat.
    for (int k = group; k < sh.rows; k += kQ * kGroups) {
      float2 sc[kQ], nm[kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) { sc[q] = both(rs[q]); nm[q] = both(-mu[q]); }
      if (k + kQ * kGroups < sh.rows) stats(row0, k + kQ * kGroups);
      else stats(row0 + gridDim.x * static_cast<long long>(sh.rows), group);
      if (k >= n) continue;
      const bool two = k + kGroups < n;
      float2 sums[kQ][2];
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        sums[q][0] = sums[q][1] = make_float2(0.0f, 0.0f);
        if (q == 1 && !two) break;
        const __nv_bfloat16* xr = reinterpret_cast<const __nv_bfloat16*>(xs + (k + q * kGroups) * x_bytes);
        const TDy* yr = reinterpret_cast<const TDy*>(ys + (k + q * kGroups) * y_bytes);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = t + v * T;
          if (c < nv) {
            float2 xh[4], dy[4], w[4];
            ln_load8(xr + 8 * c, xh);
            ln_load8(yr + 8 * c, dy);
            ln_load8(gs + 8 * c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              xh[e] = mul2(add2(xh[e], nm[q]), sc[q]);
              ag[v][e] = fma2(dy[e], xh[e], ag[v][e]);
              ab[v][e] = add2(ab[v][e], dy[e]);
              const float2 dh = mul2(dy[e], w[e]);
              sums[q][0] = add2(sums[q][0], dh);
              sums[q][1] = fma2(dh, xh[e], sums[q][1]);
            }
          }
        }
      }
      float s[2 * kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        s[2 * q] = sums[q][0].x + sums[q][0].y;
        s[2 * q + 1] = sums[q][1].x + sums[q][1].y;
      }
      ln_group_sum<T, 2 * kQ, kGroups>(s, slots, group, phase);
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        if (q == 1 && !two) break;
        const __nv_bfloat16* xr = reinterpret_cast<const __nv_bfloat16*>(xs + (k + q * kGroups) * x_bytes);
        const TDy* yr = reinterpret_cast<const TDy*>(ys + (k + q * kGroups) * y_bytes);
        __nv_bfloat16* out = dX + (row0 + k + q * kGroups) * d;
        // dx = dy g rs - rs mean(dh) - xh rs mean(dh xh)
        const float2 c1 = both(-sc[q].x * (s[2 * q] * inv_d)), c2 = both(-sc[q].x * (s[2 * q + 1] * inv_d));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = t + v * T;
          if (c < nv) {
            float2 xh[4], dy[4], w[4];
            uint32_t o[4];
            ln_load8(xr + 8 * c, xh);
            ln_load8(yr + 8 * c, dy);
            ln_load8(gs + 8 * c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              xh[e] = mul2(add2(xh[e], nm[q]), sc[q]);
              const float2 u = fma2(dy[e], mul2(w[e], sc[q]), fma2(xh[e], c2, c1));
              o[e] = pack_bf16x2(u.x, u.y);
            }
            *reinterpret_cast<uint4*>(out + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[r.stage]);
    r.next(sh.stages);
  }
  if (threadIdx.x == 0 && !ok) {         // gave up: the copies have landed before the CTA may end
    volatile uint32_t never = 0u;
    const AbortCtl quiet{&never, nullptr};
    for (long long k = filled > sh.stages ? filled - sh.stages : 0; k < filled; ++k)
      mbar_wait(&full[k % sh.stages], static_cast<uint32_t>(k / sh.stages) & 1u, quiet);
  }
  if (part == nullptr) return;                      // no gradient of g and b wanted
  // The groups of a CTA add their columns one after the other, through the ring's memory.
  float* acc_s = reinterpret_cast<float*>(ln_smem);
  float* out = part + static_cast<size_t>(blockIdx.x) * 2 * d;
  for (int k = 0; k < kGroups; ++k) {
    if (kGroups > 1) bar_sync_named<15, kLnBwdThreads>();
    if (group != k) continue;
    const bool first = k == 0, last = k == kGroups - 1;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = t + v * T;
      if (c >= nv) break;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float4 a = make_float4(ag[v][e / 2].x, ag[v][e / 2].y, ag[v][e / 2 + 1].x, ag[v][e / 2 + 1].y);
        float4 h = make_float4(ab[v][e / 2].x, ab[v][e / 2].y, ab[v][e / 2 + 1].x, ab[v][e / 2 + 1].y);
        if (!first) {
          const float4 pa = *reinterpret_cast<const float4*>(acc_s + 8 * c + e);
          const float4 ph = *reinterpret_cast<const float4*>(acc_s + d + 8 * c + e);
          a.x += pa.x; a.y += pa.y; a.z += pa.z; a.w += pa.w;
          h.x += ph.x; h.y += ph.y; h.z += ph.z; h.w += ph.w;
        }
        float* dst = last ? out : acc_s;
        *reinterpret_cast<float4*>(dst + 8 * c + e) = a;
        if (want_db) *reinterpret_cast<float4*>(dst + d + 8 * c + e) = h;
      }
    }
  }
}

// dg[j] = sum_p part[p][0][j], db[j] = sum_p part[p][1][j] in a fixed order:
// warp w of a CTA adds partials w, w + 32, ... of 128 columns, all loaded
// before the first is added, then the warps' sums are added in order.
// blockIdx.y: 0 = dg, 1 = db.
__global__ void __launch_bounds__(1024)
    layernorm_reduce_kernel(const float* __restrict__ part, int n_part, int d, float* __restrict__ dg,
                            float* __restrict__ db) {
  __shared__ float s[32][132];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 128 + 4 * lane;
  float* out = blockIdx.y == 0 ? dg : db;
  grid_dep_wait();
  if (out == nullptr) return;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (j < d)
#pragma unroll 5
    for (int p = w; p < n_part; p += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + (static_cast<size_t>(p) * 2 + blockIdx.y) * d + j);
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  *reinterpret_cast<float4*>(&s[w][4 * lane]) = a;
  __syncthreads();
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && c < d) {
    float sum = s[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 32; ++k) sum += s[k][threadIdx.x];
    out[c] = sum;
  }
}

}  // namespace lora
