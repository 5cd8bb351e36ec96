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
// 8192 rows of 4096 BF16 with residual: 43.8 us, 6.1 TB/s; 393216 rows of 128 with gate, in
// E4M3: 55.3 us, 4.6 TB/s, there bound by issued instructions, two special functions an element
// for the gate among them.  (Passes among others, each over inputs that no pass just before used;
// where two forms are compared below, calls back to back over two or three sets of inputs, which
// read up to 7% less.)
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

// kStep: elements that are moved at a time: 8 (the width is a multiple of 8, all rows lie on 16
// bytes), 4 (the same with 4 and half the bytes) or 1.  kR rows per thread: short rows share
// the weights and the reckoning of addresses.  kMin: CTAs an SM has to hold (0: no rule).
template <typename T, int kTPR, int kChunks, int kThreads, int kR, int kStep, int kMin>
__global__ void __launch_bounds__(kThreads, kMin) kda_rms_norm_kernel(const NormParams p) {
  using Raw = typename T::Raw;
  static_assert(kThreads % kTPR == 0, "whole rows");
  static_assert(kR == 1 || kTPR <= 32, "one row per thread where warps share it");
  __shared__ float s_sum[kThreads / 32], s_max[kThreads / 32];
  constexpr int kRows = kThreads / kTPR;     // rows side by side; the CTA has kR times as many
  const int j = threadIdx.x % kTPR, ric = threadIdx.x / kTPR;
  const int W = p.width;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRows * kR);
  // token and head of the CTA's first row; other rows are a few heads on
  int64_t tok0 = first;
  int32_t head0 = 0;
  if (p.heads > 1) {
    tok0 = first <= UINT32_MAX ? static_cast<uint32_t>(first) / static_cast<uint32_t>(p.heads)
                               : first / p.heads;
    head0 = static_cast<int32_t>(first - tok0 * p.heads);
  }
  // Element by element, a chunk's elements lie kGap apart and adjacent threads hold adjacent
  // elements (the 16 threads of a scale group still share its 128).  1638 rows of 4345 FP32
  // with residual and gate 33 us, with a thread's elements side by side 61.
  constexpr int kGap = kStep > 1 ? 1 : kTPR < 16 ? kTPR : 16;
  const int j0 = kE * (j - j % kGap) + j % kGap;   // the thread's first element
  const int n0 = W - j0;                      // elements from it to the row's end
  int64_t tok[kR];
  int32_t at[kR];                             // the thread's first element within its token
  int n[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int rr = r * kRows + ric;
    n[r] = first + rr < p.rows ? n0 : 0;
    tok[r] = tok0 + rr;
    at[r] = j0;
    if (p.heads > 1) {
      int32_t head = head0 + rr;
      tok[r] = tok0;
      if (p.heads >= kRows * kR) {
        if (head >= p.heads) {
          head -= p.heads;
          ++tok[r];
        }
      } else {
        const int32_t over = head / p.heads;
        tok[r] += over;
        head -= over * p.heads;
      }
      at[r] += head * W;
    }
  }
  const auto left = [&](int r, int i) { return n[r] - kE * i * kTPR; };
  const auto load = [&](Vec<T, kE> (&v)[kR][kChunks], const void* base, int64_t stride) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const Raw* q = static_cast<const Raw*>(base) + tok[r] * stride + at[r];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        if (left(r, i) > 0) v[r][i].template load_by<kStep, kGap>(q + kE * i * kTPR, left(r, i));
        else v[r][i].clear();
      }
    }
  };
  // the gate is loaded with x where registers allow, else once x and the residual are spent
  constexpr bool kGateEarly = kChunks <= 4;
  Vec<T, kE> xv[kR][kChunks], rv[kR][kChunks], gv[kR][kChunks];
  load(xv, p.x, p.xs);
  if (p.res != nullptr) load(rv, p.res, p.rs);
  if (kGateEarly && p.gate != nullptr) load(gv, p.gate, p.gs);
  float2 y[kR][kChunks][kE / 2];
  float sum[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float f[kE];
      xv[r][i].unpack(f);
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) y[r][i][e] = make_float2(f[2 * e], f[2 * e + 1]);
      if (p.res != nullptr) {
        rv[r][i].unpack(f);
#pragma unroll
        for (int e = 0; e < kE / 2; ++e)
          y[r][i][e] = add2<true>(y[r][i][e], make_float2(f[2 * e], f[2 * e + 1]));
      }
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) sq = fma2<true>(y[r][i][e], y[r][i][e], sq);
    }
    sum[r] = sq.x + sq.y;
  }
  if (!kGateEarly && p.gate != nullptr) load(gv, p.gate, p.gs);
  const auto packed = [&](int r, int i) {
    float f[kE];
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) {
      f[2 * e] = y[r][i][e].x;
      f[2 * e + 1] = y[r][i][e].y;
    }
    Vec<T, kE> o;
    o.pack(f);
    return o;
  };
  if (p.res_out != nullptr) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      Raw* q = static_cast<Raw*>(p.res_out) + tok[r] * p.ros + at[r];
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (left(r, i) > 0) packed(r, i).template store_by<kStep, kGap>(q + kE * i * kTPR, left(r, i));
    }
  }
  float rstd[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r)
    rstd[r] = rsqrtf(fmaf(row_reduce<kTPR, kThreads, false>(sum[r], s_sum, ric), p.inv_width, p.eps));

#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float2 w[kE / 2];
    if (p.weight == nullptr) {
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) w[e] = make_float2(1.f, 1.f);
    } else {
      const int nw = n0 - kE * i * kTPR;
      Vec<F32, kE> wv;
      if (nw > 0) wv.template load_by<kStep, kGap>(p.weight + j0 + kE * i * kTPR, nw);
      else wv.clear();
#pragma unroll
      for (int e = 0; e < kE / 2; ++e)
        w[e] = make_float2(__uint_as_float(wv.w[2 * e]), __uint_as_float(wv.w[2 * e + 1]));
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
      for (int e = 0; e < kE / 2; ++e)
        y[r][i][e] = mul2<true>(mul2<true>(y[r][i][e], make_float2(rstd[r], rstd[r])), w[e]);
      if (p.gate != nullptr) {
        float g[kE];
        gv[r][i].unpack(g);
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) {
          const float2 z = make_float2(g[2 * e], g[2 * e + 1]);
          y[r][i][e] = mul2<true>(y[r][i][e], sigmoid2(z));
          if (!p.sigmoid) y[r][i][e] = mul2<true>(y[r][i][e], z);
        }
      }
    }
  }

  if (!p.out8) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      Raw* q = static_cast<Raw*>(p.out) + (first + r * kRows + ric) * W + j0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (left(r, i) > 0) packed(r, i).template store_by<kStep, kGap>(q + kE * i * kTPR, left(r, i));
    }
    return;
  }

  // 8 bits.  Scale and value / scale are the quotients, rounded once: estimate, what it leaves of
  // the dividend, and that times the reciprocal on top.  (With products by 448 / max, within 2^-22,
  // codes next to a border of E4M3 went to the other side.)
  const auto quotient_448 = [](float amax) {
    const float q = amax * (1.f / kE4m3Max);
    const float r = fmaf(fmaf(-q, kE4m3Max, amax), 1.f / kE4m3Max, q);
    return fabsf(amax) < INFINITY ? r : amax;
  };
  const auto amax_of = [&](int r, int i) {
    float m = max_nan(fabsf(y[r][i][0].x), fabsf(y[r][i][0].y));
#pragma unroll
    for (int e = 1; e < kE / 2; ++e)
      m = max_nan(m, max_nan(fabsf(y[r][i][e].x), fabsf(y[r][i][e].y)));
    return m;
  };
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int64_t row = first + r * kRows + ric;
    float scale[kChunks];
    if (p.group == 0) {
      float m = amax_of(r, 0);
#pragma unroll
      for (int i = 1; i < kChunks; ++i) m = max_nan(m, amax_of(r, i));
      const float amax = max_nan(row_reduce<kTPR, kThreads, true>(m, s_max, ric), kAmaxFloor);
      const float sc = quotient_448(amax);
      if (n[r] > 0 && j == 0) p.scales[row] = sc;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) scale[i] = sc;
    } else if constexpr (kTPR % 16 == 0) {     // (shorter rows are one group)
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        float m = amax_of(r, i);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        scale[i] = quotient_448(max_nan(m, kAmaxFloor));
        if (left(r, i) > 0 && (j & 15) == 0)
          p.scales[row * p.groups + (j + i * kTPR) / 16] = scale[i];
      }
    }
    uint8_t* o = static_cast<uint8_t*>(p.out) + row * W + j0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      // (over an infinite scale a number is 0 and an infinity has no value)
      const float inv = rcp_approx(scale[i]), div = scale[i] < INFINITY ? -scale[i] : 0.f;
      const auto quotient = [&](float2 v) {
        const float2 f = make_float2(inv, inv), e = mul2<true>(v, f);
        return fma2<true>(fma2<true>(e, make_float2(div, div), v), f, e);
      };
      uint32_t q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 a = quotient(y[r][i][2 * h]), b = quotient(y[r][i][2 * h + 1]);
        q[h] = e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16);
      }
      if constexpr (kStep == 8) {
        if (left(r, i) > 0) *reinterpret_cast<uint2*>(o + kE * i * kTPR) = make_uint2(q[0], q[1]);
      } else if constexpr (kStep == 4) {
        if (left(r, i) > 0) *reinterpret_cast<uint32_t*>(o + kE * i * kTPR) = q[0];
        if (left(r, i) > 4) *reinterpret_cast<uint32_t*>(o + kE * i * kTPR + 4) = q[1];
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (e * kGap < left(r, i))
            o[kE * i * kTPR + e * kGap] = static_cast<uint8_t>(q[e / 4] >> (8 * (e % 4)));
      }
    }
  }
}

template <typename T, int kTPR, int kChunks, int kThreads, int kR, int kStep, int kMin = 0>
bool go_step(const NormParams& p, cudaStream_t s) {
  const int64_t per = kThreads / kTPR * kR, grid = (p.rows + per - 1) / per;
  if (grid > INT32_MAX) return false;
  kda_rms_norm_kernel<T, kTPR, kChunks, kThreads, kR, kStep, kMin>
      <<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
  return true;
}
template <typename T, int kTPR, int kChunks, int kThreads, int kR = 1>
bool go(const NormParams& p, cudaStream_t s) {
  if (p.step == 8) return go_step<T, kTPR, kChunks, kThreads, kR, 8>(p, s);
  if (p.step == 4) return go_step<T, kTPR, kChunks, kThreads, kR, 4>(p, s);
  return go_step<T, kTPR, kChunks, kThreads, kR, 1>(p, s);
}

template <typename T>
bool launch(NormParams p, cudaStream_t s) {
  // The fewest threads whose registers hold the row in few chunks each.
  const int W = p.width;
  if (W <= 128) p.group = 0;      // one scale group: the row
  if (W <= 64) return go<T, 8, 1, 128, 4>(p, s);
  // Rows of 65 to 128: two chunks a thread, which spend less on addresses and sums than one.  16-bit
  // types: two rows of them in 64 registers (393216 rows of 128 BF16, us: with gate in E4M3 51.7,
  // 53.8 without that limit, one chunk of two rows 64.0; the bare norm 37.4, 39.0, 44.1).  FP32 rows
  // take twice the registers, and under that limit 436 bytes a thread went to memory and back: one
  // row (294912 rows of 128, us, one row / two in 64 registers / two without a limit: bare 49.7 /
  // 51.7 / 51.7, with residual and gate 114 / 175 / 115, gate in E4M3 53.8 / 71.5 / 57.8).  Element
  // by element one chunk is better (48000 rows of 125: 14.6 against 18.4).
  if (W <= 128) {
    if (p.step == 1) return go_step<T, 16, 1, 128, 2, 1>(p, s);
    if constexpr (sizeof(typename T::Raw) == 4) {
      if (p.step == 8) return go_step<T, 8, 2, 128, 1, 8>(p, s);
      return go_step<T, 8, 2, 128, 1, 4>(p, s);
    } else {
      if (p.step == 8) return go_step<T, 8, 2, 128, 2, 8, 8>(p, s);
      return go_step<T, 8, 2, 128, 2, 4, 8>(p, s);
    }
  }
  if (W <= 256) return go<T, 32, 1, 128, 2>(p, s);
  if (W <= 512) return go<T, 32, 2, 128>(p, s);
  if (W <= 1024) return go<T, 128, 1, 128>(p, s);
  if (W <= 2048) return go<T, 128, 2, 128>(p, s);
  if (W <= 4096) return go<T, 256, 2, 256>(p, s);
  if (W <= 8192) return go<T, 256, 4, 256>(p, s);
  if (W <= 16384) return go<T, 512, 4, 512>(p, s);
  // (FP32 rows leave 176 bytes a thread and more in memory here; 1024 threads of half as much have
  // 64 registers and lose more: 1024 rows of 32768 89 against 121 us, with residual 122 against 177)
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
