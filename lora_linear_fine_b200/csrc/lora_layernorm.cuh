// lora_layernorm.cuh — layer norm with trained scale and shift, forward and
// backward, beside the RMSNorm prologue (lora_norm_rope.cuh).
//
//   mean = sum_j x_j / d,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / d + eps)
//   xh = (x - mean) rstd,  y = xh g + b                           (per token)
//   dh = dy g,  dx = rstd (dh - mean_j(dh) - xh mean_j(dh xh))
//   dg = sum_m dy xh,  db = sum_m dy
//
// A row is held in the registers of a group of T threads (two 16-byte chunks,
// 16 features, a thread), so it is read from memory once: the forward takes
// the mean and then the squares around it from registers, the backward both
// of its means at once.  Groups of T = 32 ... 256 threads share a CTA of 256;
// wider rows take a CTA each.  T is the smallest that holds the row: fewer
// threads a row would need a second pass, more would leave lanes idle and
// lengthen the reduction.
//
// The backward's CTAs stay for all their rows and keep dg and db of their
// columns in registers; they write one partial row each at the end, and
// layernorm_reduce_kernel adds the partials in a fixed order, so the
// gradients of one problem on one device are the same bits in every call.
#pragma once

#include "lora_norm_rope.cuh"

namespace lora {

constexpr int kLnMaxD = 16384;       // 1024 threads x 16 features
constexpr int kLnNV = 2;             // 16-byte chunks a thread

template <int T>
struct LnCfg {
  static constexpr int kThreads = T > 256 ? T : 256;
  static constexpr int kGroups = kThreads / T;     // rows a CTA works on at a time
  static constexpr int kWarps = T / 32;            // warps a row
};

// Sums of `n` values over the T threads of a group, the same in every thread:
// a butterfly within the warps, the warps' sums through `slots` (one row of
// kWarps x n floats a group, alternating between two rows so that one barrier
// a call is enough).
template <int T, int n>
__device__ __forceinline__ void ln_group_sum(float (&v)[n], float* slots, int group, uint32_t& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    const int w = (threadIdx.x % T) >> 5, lane = threadIdx.x & 31;
    float* s = slots + ((phase & 1u) * LnCfg<T>::kGroups + group) * (W * 2);
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

template <int T>
__global__ void __launch_bounds__(LnCfg<T>::kThreads)
    layernorm_fwd_kernel(const __nv_bfloat16* X, const __nv_bfloat16* __restrict__ g,
                         const __nv_bfloat16* __restrict__ b, long long M, int d, float eps,
                         __nv_bfloat16* Y, float* __restrict__ mean, float* __restrict__ rstd) {
  using C = LnCfg<T>;
  __shared__ float slots[2 * C::kGroups * C::kWarps * 2];
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  const int nv = d / 8;
  const float inv_d = 1.0f / static_cast<float>(d);
  uint32_t phase = 0;
  grid_dep_wait();
  for (long long row = blockIdx.x * static_cast<long long>(C::kGroups) + group; row < M;
       row += static_cast<long long>(gridDim.x) * C::kGroups) {
    const uint4* xr = reinterpret_cast<const uint4*>(X + row * d);
    float x[kLnNV][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      unpack_bf16x8(c < nv ? xr[c] : make_uint4(0u, 0u, 0u, 0u), x[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[v][e];
    }
    ln_group_sum<T, 1>(s, slots, group, phase);
    const float mu = s[0] * inv_d;
    s[0] = 0.0f;
#pragma unroll
    for (int v = 0; v < kLnNV; ++v)
      if (t + v * T < nv)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(x[v][e] - mu, x[v][e] - mu, s[0]);
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
      float w[8], sh[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(g) + c), w);
      unpack_bf16x8(b != nullptr ? __ldg(reinterpret_cast<const uint4*>(b) + c) : make_uint4(0u, 0u, 0u, 0u), sh);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf((x[v][e] - mu) * rs, w[e], sh[e]);
      yr[c] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                         pack_bf16x2(y[6], y[7]));
    }
  }
}

__device__ __forceinline__ void ln_load8(const __nv_bfloat16* p, float (&f)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void ln_load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// part [gridDim.x][2][d] fp32: each CTA's dg and db over its rows.
template <int T, typename TDy>
__global__ void __launch_bounds__(LnCfg<T>::kThreads)
    layernorm_bwd_kernel(const TDy* dY, const __nv_bfloat16* X,
                         const __nv_bfloat16* __restrict__ g, const float* __restrict__ mean,
                         const float* __restrict__ rstd, long long M, int d, __nv_bfloat16* dX,
                         float* __restrict__ part) {
  using C = LnCfg<T>;
  extern __shared__ float acc_s[];                  // [2][d] when several groups share the CTA
  __shared__ float slots[2 * C::kGroups * C::kWarps * 2];
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  const int nv = d / 8;
  const float inv_d = 1.0f / static_cast<float>(d);
  uint32_t phase = 0;
  float ag[kLnNV][8] = {}, ab[kLnNV][8] = {};
  grid_dep_wait();
  for (long long row = blockIdx.x * static_cast<long long>(C::kGroups) + group; row < M;
       row += static_cast<long long>(gridDim.x) * C::kGroups) {
    const float mu = mean[row], rs = rstd[row];
    float xh[kLnNV][8], dh[kLnNV][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      if (c < nv) {
        float w[8];
        unpack_bf16x8(*reinterpret_cast<const uint4*>(X + row * d + 8 * c), xh[v]);
        ln_load8(dY + row * d + 8 * c, dh[v]);
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(g) + c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[v][e] = (xh[v][e] - mu) * rs;
          ag[v][e] = fmaf(dh[v][e], xh[v][e], ag[v][e]);
          ab[v][e] += dh[v][e];
          dh[v][e] *= w[e];
          s[0] += dh[v][e];
          s[1] = fmaf(dh[v][e], xh[v][e], s[1]);
        }
      }
    }
    ln_group_sum<T, 2>(s, slots, group, phase);
    const float c1 = s[0] * inv_d, c2 = s[1] * inv_d;
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      if (c < nv) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rs * (dh[v][e] - c1 - xh[v][e] * c2);
        *reinterpret_cast<uint4*>(dX + row * d + 8 * c) =
            make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                       pack_bf16x2(o[6], o[7]));
      }
    }
  }
  if (part == nullptr) return;                      // no gradient of g and b wanted
  // The groups of a CTA add their columns one after the other.
  float* out = part + static_cast<size_t>(blockIdx.x) * 2 * d;
  for (int k = 0; k < C::kGroups; ++k) {
    if (C::kGroups > 1) __syncthreads();
    if (group != k) continue;
    const bool first = k == 0, last = k == C::kGroups - 1;
#pragma unroll
    for (int v = 0; v < kLnNV; ++v) {
      const int c = t + v * T;
      if (c >= nv) break;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float4 a = make_float4(ag[v][e], ag[v][e + 1], ag[v][e + 2], ag[v][e + 3]);
        float4 h = make_float4(ab[v][e], ab[v][e + 1], ab[v][e + 2], ab[v][e + 3]);
        if (!first) {
          const float4 pa = *reinterpret_cast<const float4*>(acc_s + 8 * c + e);
          const float4 ph = *reinterpret_cast<const float4*>(acc_s + d + 8 * c + e);
          a.x += pa.x; a.y += pa.y; a.z += pa.z; a.w += pa.w;
          h.x += ph.x; h.y += ph.y; h.z += ph.z; h.w += ph.w;
        }
        float* dst = last ? out : acc_s;
        *reinterpret_cast<float4*>(dst + 8 * c + e) = a;
        *reinterpret_cast<float4*>(dst + d + 8 * c + e) = h;
      }
    }
  }
}

// dg[j] = sum_p part[p][0][j], db[j] = sum_p part[p][1][j] in a fixed order:
// warp w of a CTA adds partials w, w + 8, ... of 32 columns, then the warps'
// sums are added in order.  blockIdx.y: 0 = dg, 1 = db.
__global__ void __launch_bounds__(256)
    layernorm_reduce_kernel(const float* __restrict__ part, int n_part, int d, float* __restrict__ dg,
                            float* __restrict__ db) {
  __shared__ float s[8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 32 + lane;
  float* out = blockIdx.y == 0 ? dg : db;
  grid_dep_wait();
  if (out == nullptr) return;
  float a = 0.0f;
  if (j < d)
    for (int p = w; p < n_part; p += 8) a += part[(static_cast<size_t>(p) * 2 + blockIdx.y) * d + j];
  s[w][lane] = a;
  __syncthreads();
  if (w == 0 && j < d) {
    for (int k = 1; k < 8; ++k) a += s[k][lane];
    out[j] = a;
  }
}

}  // namespace lora
