// kda_norm.cu — root-mean-square norm of rows, with the residual's addition before it and a
// gate after it, written in the rows' type or in E4M3 with FP32 scales.
//
//   r = x + residual;  y = r / sqrt(mean(r^2) + eps) * weight * act(gate)
//   8 bits: scale = max(max|y|, 2^-40) / 448 per group, out = e4m3(y / scale)
//
// Every element is read once and written once and kept in registers between the two row
// sums; nothing else is to be done, so the bound is HBM for many rows and the latency of
// one load, two reductions and one store for few.  r is not rounded before the norm (the
// stored residual is its rounding): one rounding fewer than norming the stored sum.
//
// kTPR threads share a row: a part of a warp for short rows (the heads of a token: no
// barrier at all), several warps for long ones (one barrier per reduction).  A thread holds
// kChunks chunks of 8 elements, chunk i of thread j at element 8 (j + i kTPR), so that 16
// adjacent threads hold 128 adjacent elements: a scale group is a half-warp reduction.
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace norm {

constexpr int kE = 8;               // elements per chunk
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 9.094947017729282e-13f;   // 2^-40

// maximum that keeps a NaN, as the scale of a group with a NaN must be one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// two E4M3 bytes, rounded to nearest even, saturating; a in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int kTPR, int kThreads, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* smem, int row_in_cta) {
  constexpr int kIn = kTPR < 32 ? kTPR : 32;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  if constexpr (kTPR > 32) {
    constexpr int kWarps = kTPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) smem[warp] = v;
    __syncthreads();
    v = smem[row_in_cta * kWarps];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      const float w = smem[row_in_cta * kWarps + i];
      v = kMax ? max_nan(v, w) : v + w;
    }
  }
  return v;
}

template <typename T, int kTPR, int kChunks, int kThreads>
__global__ void __launch_bounds__(kThreads) kda_rms_norm_kernel(const NormParams p) {
  using Raw = typename T::Raw;
  static_assert(kThreads % kTPR == 0 && kTPR % 16 == 0, "whole rows and scale groups");
  __shared__ float s_sum[kThreads / 32], s_max[kThreads / 32];
  const int j = threadIdx.x % kTPR, ric = threadIdx.x / kTPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / kTPR) + ric;
  const bool live = row < p.rows;
  const int64_t tok = row / p.heads;
  const int32_t head_off = static_cast<int32_t>(row - tok * p.heads) * p.width;
  const int W = p.width;

  // Loaded with x where registers allow, else once x and the residual are spent.
  constexpr bool kGateEarly = kChunks <= 4;
  Vec<T, kE> xv[kChunks], rv[kChunks], gv[kChunks];
  auto load_gate = [&] {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = kE * (j + i * kTPR);
      const int n = live ? W - c : 0;
      const Raw* gp = static_cast<const Raw*>(p.gate) + tok * p.gs + head_off + c;
      if (n > 0) gv[i].load(gp, p.vec, n);
      else gv[i].clear();
    }
  };
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = kE * (j + i * kTPR);
    const int n = live ? W - c : 0;
    const Raw* xp = static_cast<const Raw*>(p.x) + tok * p.xs + head_off + c;
    if (n > 0) xv[i].load(xp, p.vec, n);
    else xv[i].clear();
    if (p.res != nullptr) {
      const Raw* rp = static_cast<const Raw*>(p.res) + tok * p.rs + head_off + c;
      if (n > 0) rv[i].load(rp, p.vec, n);
      else rv[i].clear();
    }
  }
  if (kGateEarly && p.gate != nullptr) load_gate();
  float y[kChunks][kE];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    xv[i].unpack(y[i]);
    if (p.res != nullptr) {
      float f[kE];
      rv[i].unpack(f);
#pragma unroll
      for (int e = 0; e < kE; ++e) y[i][e] += f[e];
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) sum = fmaf(y[i][e], y[i][e], sum);
  }
  if (!kGateEarly && p.gate != nullptr) load_gate();
  if (p.res_out != nullptr) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = kE * (j + i * kTPR);
      const int n = live ? W - c : 0;
      Vec<T, kE> o;
      o.pack(y[i]);
      if (n > 0)
        o.store(static_cast<Raw*>(p.res_out) + tok * p.ros + head_off + c, p.vec, n);
    }
  }
  sum = row_reduce<kTPR, kThreads, false>(sum, s_sum, ric);
  const float rstd = rsqrtf(sum / static_cast<float>(W) + p.eps);

#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = kE * (j + i * kTPR);
    const int n = W - c;
    float w[kE];
    if (p.weight == nullptr) {
#pragma unroll
      for (int e = 0; e < kE; ++e) w[e] = 1.f;
    } else {
      Vec<F32, kE> wv;
      if (n > 0) wv.load(p.weight + c, p.vec_w, n);
      else wv.clear();
      wv.unpack(w);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) y[i][e] *= rstd * w[e];
    if (p.gate != nullptr) {
      float g[kE];
      gv[i].unpack(g);
#pragma unroll
      for (int e = 0; e < kE; ++e) y[i][e] *= p.sigmoid ? sigmoid(g[e]) : silu(g[e]);
    }
  }

  if (!p.out8) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = kE * (j + i * kTPR);
      const int n = live ? W - c : 0;
      Vec<T, kE> o;
      o.pack(y[i]);
      if (n > 0)
        o.store(static_cast<Raw*>(p.out) + row * W + c, p.vec, n);
    }
    return;
  }

  float inv[kChunks];
  if (p.group == 0) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) m = max_nan(m, fabsf(y[i][e]));
    const float amax = max_nan(row_reduce<kTPR, kThreads, true>(m, s_max, ric), kAmaxFloor);
    if (live && j == 0) p.scales[row] = amax / kE4m3Max;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) inv[i] = kE4m3Max / amax;
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) m = max_nan(m, fabsf(y[i][e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float amax = max_nan(m, kAmaxFloor);
      const int c = kE * (j + i * kTPR);
      if (live && (j & 15) == 0 && c < W) p.scales[row * p.groups + c / 128] = amax / kE4m3Max;
      inv[i] = kE4m3Max / amax;
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = kE * (j + i * kTPR);
    const int n = live ? W - c : 0;
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      q[h] = e4m3x2(y[i][4 * h] * inv[i], y[i][4 * h + 1] * inv[i]) |
             (e4m3x2(y[i][4 * h + 2] * inv[i], y[i][4 * h + 3] * inv[i]) << 16);
    uint8_t* o = static_cast<uint8_t*>(p.out) + row * W + c;
    if (n >= kE && p.vec) {
      *reinterpret_cast<uint2*>(o) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (e < n) o[e] = static_cast<uint8_t>(q[e / 4] >> (8 * (e % 4)));
    }
  }
}

template <typename T>
bool launch(const NormParams& p, cudaStream_t s) {
  const auto go = [&](auto kernel, int tpr, int threads) {
    const int64_t per = threads / tpr, grid = (p.rows + per - 1) / per;
    if (grid > INT32_MAX) return false;
    kernel<<<static_cast<unsigned>(grid), threads, 0, s>>>(p);
    return true;
  };
  // The fewest threads whose registers hold the row in few chunks each.
  const int W = p.width;
  if (W <= 128) return go(kda_rms_norm_kernel<T, 16, 1, 128>, 16, 128);
  if (W <= 256) return go(kda_rms_norm_kernel<T, 32, 1, 128>, 32, 128);
  if (W <= 512) return go(kda_rms_norm_kernel<T, 32, 2, 128>, 32, 128);
  if (W <= 1024) return go(kda_rms_norm_kernel<T, 128, 1, 128>, 128, 128);
  if (W <= 2048) return go(kda_rms_norm_kernel<T, 128, 2, 128>, 128, 128);
  if (W <= 4096) return go(kda_rms_norm_kernel<T, 256, 2, 256>, 256, 256);
  if (W <= 8192) return go(kda_rms_norm_kernel<T, 256, 4, 256>, 256, 256);
  if (W <= 16384) return go(kda_rms_norm_kernel<T, 512, 4, 512>, 512, 512);
  return go(kda_rms_norm_kernel<T, 512, 8, 512>, 512, 512);
}

}  // namespace norm

bool launch_norm(const NormParams& p, int dtype, cudaStream_t s) {
  if (dtype == 0) return norm::launch<Bf16>(p, s);
  if (dtype == 1) return norm::launch<F16>(p, s);
  return norm::launch<F32>(p, s);
}

}  // namespace layer
}  // namespace kda
