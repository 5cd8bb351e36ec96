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

// kVec: the width is a multiple of 8 and all rows may be moved 16 bytes at a time.
template <typename T, int kTPR, int kChunks, int kThreads, bool kVec>
__global__ void __launch_bounds__(kThreads) kda_rms_norm_kernel(const NormParams p) {
  using Raw = typename T::Raw;
  static_assert(kThreads % kTPR == 0 && kTPR % 16 == 0, "whole rows and scale groups");
  __shared__ float s_sum[kThreads / 32], s_max[kThreads / 32];
  constexpr int kRows = kThreads / kTPR;
  const int j = threadIdx.x % kTPR, ric = threadIdx.x / kTPR;
  const int W = p.width;
  // token and head of the row: one division for the CTA's first row, where heads allow it
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows, row = first + ric;
  int64_t tok = row;
  int32_t head = 0;
  if (p.heads > 1) {
    const bool small = first <= UINT32_MAX;
    tok = small ? static_cast<uint32_t>(first) / static_cast<uint32_t>(p.heads) : first / p.heads;
    head = static_cast<int32_t>(first - tok * p.heads) + ric;
    if (p.heads >= kRows) {
      if (head >= p.heads) {
        head -= p.heads;
        ++tok;
      }
    } else {
      const int32_t over = head / p.heads;
      tok += over;
      head -= over * p.heads;
    }
  }
  const int32_t at = head * W + kE * j;      // first element of the thread, within its token
  int n = row < p.rows ? W - kE * j : 0;     // elements from there to the end of the row
  const auto left = [&](int i) { return n - kE * i * kTPR; };

  const auto load = [&](Vec<T, kE> (&v)[kChunks], const void* base, int64_t stride) {
    const Raw* q = static_cast<const Raw*>(base) + tok * stride + at;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (left(i) > 0) v[i].template load<kVec>(q + kE * i * kTPR, left(i));
      else v[i].clear();
    }
  };
  // the gate is loaded with x where registers allow, else once x and the residual are spent
  constexpr bool kGateEarly = kChunks <= 4;
  Vec<T, kE> xv[kChunks], rv[kChunks], gv[kChunks];
  load(xv, p.x, p.xs);
  if (p.res != nullptr) load(rv, p.res, p.rs);
  if (kGateEarly && p.gate != nullptr) load(gv, p.gate, p.gs);
  float2 y[kChunks][kE / 2];
  float2 sq = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float f[kE];
    xv[i].unpack(f);
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) y[i][e] = make_float2(f[2 * e], f[2 * e + 1]);
    if (p.res != nullptr) {
      rv[i].unpack(f);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e)
        y[i][e] = add2<true>(y[i][e], make_float2(f[2 * e], f[2 * e + 1]));
    }
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) sq = fma2<true>(y[i][e], y[i][e], sq);
  }
  if (!kGateEarly && p.gate != nullptr) load(gv, p.gate, p.gs);
  const auto packed = [&](int i) {
    float f[kE];
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) {
      f[2 * e] = y[i][e].x;
      f[2 * e + 1] = y[i][e].y;
    }
    Vec<T, kE> o;
    o.pack(f);
    return o;
  };
  if (p.res_out != nullptr) {
    Raw* q = static_cast<Raw*>(p.res_out) + tok * p.ros + at;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (left(i) > 0) packed(i).template store<kVec>(q + kE * i * kTPR, left(i));
  }
  const float sum = row_reduce<kTPR, kThreads, false>(sq.x + sq.y, s_sum, ric);
  const float rstd = rsqrtf(fmaf(sum, p.inv_width, p.eps));

#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    if (p.weight == nullptr) {
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) y[i][e] = mul2<true>(y[i][e], make_float2(rstd, rstd));
    } else {
      // (of a thread without a row too: its products are not written)
      const int nw = W - kE * (j + i * kTPR);
      Vec<F32, kE> wv;
      if (nw > 0) wv.template load<kVec>(p.weight + kE * (j + i * kTPR), nw);
      else wv.clear();
#pragma unroll
      for (int e = 0; e < kE / 2; ++e)
        y[i][e] = mul2<true>(mul2<true>(y[i][e], make_float2(rstd, rstd)),
                             make_float2(__uint_as_float(wv.w[2 * e]),
                                         __uint_as_float(wv.w[2 * e + 1])));
    }
    if (p.gate != nullptr) {
      float g[kE];
      gv[i].unpack(g);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        const float2 z = make_float2(g[2 * e], g[2 * e + 1]);
        y[i][e] = mul2<true>(y[i][e], sigmoid2(z));
        if (!p.sigmoid) y[i][e] = mul2<true>(y[i][e], z);
      }
    }
  }

  if (!p.out8) {
    Raw* q = static_cast<Raw*>(p.out) + row * W + kE * j;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (left(i) > 0) packed(i).template store<kVec>(q + kE * i * kTPR, left(i));
    return;
  }

  // 8 bits.  The scale and the factor 1 / scale are products with rounded constants and the
  // reciprocal approximation: within 2^-22 of the quotients.
  const auto amax_of = [&](int i) {
    float m = max_nan(fabsf(y[i][0].x), fabsf(y[i][0].y));
#pragma unroll
    for (int e = 1; e < kE / 2; ++e) m = max_nan(m, max_nan(fabsf(y[i][e].x), fabsf(y[i][e].y)));
    return m;
  };
  float factor[kChunks];
  if (p.group == 0) {
    float m = amax_of(0);
#pragma unroll
    for (int i = 1; i < kChunks; ++i) m = max_nan(m, amax_of(i));
    const float amax = max_nan(row_reduce<kTPR, kThreads, true>(m, s_max, ric), kAmaxFloor);
    if (n > 0 && j == 0) p.scales[row] = amax * (1.f / kE4m3Max);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) factor[i] = kE4m3Max * rcp_approx(amax);
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float m = amax_of(i);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float amax = max_nan(m, kAmaxFloor);
      if (left(i) > 0 && (j & 15) == 0)
        p.scales[row * p.groups + (j + i * kTPR) / 16] = amax * (1.f / kE4m3Max);
      factor[i] = kE4m3Max * rcp_approx(amax);
    }
  }
  uint8_t* o = static_cast<uint8_t*>(p.out) + row * W + kE * j;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const float2 f = make_float2(factor[i], factor[i]);
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 a = mul2<true>(y[i][2 * h], f), b = mul2<true>(y[i][2 * h + 1], f);
      q[h] = e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16);
    }
    if constexpr (kVec) {
      if (left(i) > 0) *reinterpret_cast<uint2*>(o + kE * i * kTPR) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (e < left(i)) o[kE * i * kTPR + e] = static_cast<uint8_t>(q[e / 4] >> (8 * (e % 4)));
    }
  }
}

template <typename T, int kTPR, int kChunks, int kThreads>
bool go(const NormParams& p, cudaStream_t s) {
  const int64_t per = kThreads / kTPR, grid = (p.rows + per - 1) / per;
  if (grid > INT32_MAX) return false;
  const auto kernel = p.vec ? kda_rms_norm_kernel<T, kTPR, kChunks, kThreads, true>
                            : kda_rms_norm_kernel<T, kTPR, kChunks, kThreads, false>;
  kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
  return true;
}

template <typename T>
bool launch(const NormParams& p, cudaStream_t s) {
  // The fewest threads whose registers hold the row in few chunks each.
  const int W = p.width;
  if (W <= 128) return go<T, 16, 1, 128>(p, s);
  if (W <= 256) return go<T, 32, 1, 128>(p, s);
  if (W <= 512) return go<T, 32, 2, 128>(p, s);
  if (W <= 1024) return go<T, 128, 1, 128>(p, s);
  if (W <= 2048) return go<T, 128, 2, 128>(p, s);
  if (W <= 4096) return go<T, 256, 2, 256>(p, s);
  if (W <= 8192) return go<T, 256, 4, 256>(p, s);
  if (W <= 16384) return go<T, 512, 4, 512>(p, s);
  return go<T, 512, 8, 512>(p, s);
}

}  // namespace norm

bool launch_norm(const NormParams& p, int dtype, cudaStream_t s) {
  if (dtype == 0) return norm::launch<Bf16>(p, s);
  if (dtype == 1) return norm::launch<F16>(p, s);
  return norm::launch<F32>(p, s);
}

}  // namespace layer
}  // namespace kda
