// kda_layer.cuh — launch parameters and device helpers shared by the layer operators
// (short convolution, selective scan, norm; include/kda_layer.h) and their host code.
#pragma once
#include <cstdint>

#include "kda_common.cuh"
#include "sm100_primitives.cuh"

namespace kda {
namespace layer {

constexpr int32_t kStatusBadIndex = 19;   // KDA_ERR_BAD_STATE_INDEX

// ---- element types -------------------------------------------------------------------
// A tag per activation type: its storage and its exact conversion to and rounding from FP32.
struct Bf16 {
  using Raw = uint16_t;
  static __device__ __forceinline__ float to(Raw r) { return bf16_to_f32(r); }
  static __device__ __forceinline__ Raw from(float f) {
    return static_cast<Raw>(pack_bf16(f, 0.f) & 0xffffu);
  }
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) { return pack_bf16(a, b); }
};
struct F16 {
  using Raw = uint16_t;
  static __device__ __forceinline__ float to(Raw r) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(r));
    return f;
  }
  static __device__ __forceinline__ Raw from(float f) {
    return static_cast<Raw>(pack_f16(f, 0.f) & 0xffffu);
  }
  static __device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(to(static_cast<Raw>(w & 0xffffu)), to(static_cast<Raw>(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) { return pack_f16(a, b); }
};
struct F32 {
  using Raw = float;
  static __device__ __forceinline__ float to(Raw r) { return r; }
  static __device__ __forceinline__ Raw from(float f) { return f; }
};

// n adjacent elements as 32-bit words.  kVec: the address is a multiple of the vector's size
// (at most 16 bytes) and all n elements are there, a property of the whole launch; else
// element by element up to `count`: elements past it read as 0 and are not written.
template <typename T, int n>
struct Vec {
  static constexpr int kBytes = n * static_cast<int>(sizeof(typename T::Raw));
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  // Not kVec: element by element, kGap apart, those below `count`.
  template <bool kVec, int kGap = 1>
  __device__ __forceinline__ void load(const typename T::Raw* p, int count = n) {
    if constexpr (kVec) {
      if constexpr (kBytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(p)[i];
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      } else if constexpr (kBytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
      } else if constexpr (kBytes == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        w[0] = *reinterpret_cast<const uint16_t*>(p);
      }
    } else {
      clear();
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i * kGap < count) {
          if constexpr (sizeof(typename T::Raw) == 4)
            w[i] = __float_as_uint(p[i * kGap]);
          else
            w[i / 2] |= static_cast<uint32_t>(p[i * kGap]) << (16 * (i % 2));
        }
    }
  }
  template <bool kVec, int kGap = 1>
  __device__ __forceinline__ void store(typename T::Raw* p, int count = n) const {
    if constexpr (kVec) {
      if constexpr (kBytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(p)[i] =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t*>(p) = w[0];
      } else {
        *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i * kGap < count) {
          if constexpr (sizeof(typename T::Raw) == 4)
            p[i * kGap] = __uint_as_float(w[i]);
          else
            p[i * kGap] = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
        }
    }
  }
  // In pieces of kStep elements that lie whole within `count` or behind it (kStep = 1: any,
  // kGap apart).
  template <int kStep, int kGap = 1>
  __device__ __forceinline__ void load_by(const typename T::Raw* p, int count) {
    if constexpr (kStep == n) {
      load<true>(p);
    } else if constexpr (kStep == 1) {
      load<false, kGap>(p, count);
    } else {
#pragma unroll
      for (int i = 0; i < n / kStep; ++i) {
        Vec<T, kStep> v;
        if (i * kStep < count) v.template load<true>(p + i * kStep);
        else v.clear();
#pragma unroll
        for (int k = 0; k < kWords * kStep / n; ++k) w[i * (kWords * kStep / n) + k] = v.w[k];
      }
    }
  }
  template <int kStep, int kGap = 1>
  __device__ __forceinline__ void store_by(typename T::Raw* p, int count) const {
    if constexpr (kStep == n) {
      store<true>(p);
    } else if constexpr (kStep == 1) {
      store<false, kGap>(p, count);
    } else {
#pragma unroll
      for (int i = 0; i < n / kStep; ++i) {
        Vec<T, kStep> v;
#pragma unroll
        for (int k = 0; k < kWords * kStep / n; ++k) v.w[k] = w[i * (kWords * kStep / n) + k];
        if (i * kStep < count) v.template store<true>(p + i * kStep);
      }
    }
  }
  __device__ __forceinline__ void unpack(float (&f)[n]) const {
    if constexpr (sizeof(typename T::Raw) == 4) {
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (n == 1) {
      f[0] = T::to(static_cast<uint16_t>(w[0]));
    } else {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float2 v = T::unpack2(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[n]) {
    if constexpr (sizeof(typename T::Raw) == 4) {
#pragma unroll
      for (int i = 0; i < n; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (n == 1) {
      w[0] = T::from(f[0]);
    } else {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) w[i] = T::pack2(f[2 * i], f[2 * i + 1]);
    }
  }
};

// ---- arithmetic ----------------------------------------------------------------------
// 1 / (1 + e^-x); the reciprocal of an infinite denominator is 0, the limit
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + ex2(-x * kLog2e)); }
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 t = mul2<true>(x, make_float2(-kLog2e, -kLog2e));
  const float2 d = add2<true>(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
__device__ __forceinline__ float2 silu2(float2 x) { return mul2<true>(x, sigmoid2(x)); }

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---- sequences -----------------------------------------------------------------------
// Row range of sequence n, from device metadata of either integer type, clamped to
// [0, rows] whatever it holds.
struct Seqs {
  const void* cu;      // NULL: equal lengths of fixed_len rows
  int32_t cu64;        // the entries are INT64
  int32_t num, rows, fixed_len;

  __device__ __forceinline__ int32_t start(int32_t n) const {
    if (cu == nullptr) return n * fixed_len;
    if (cu64) {
      const int64_t a = static_cast<const int64_t*>(cu)[n];
      return static_cast<int32_t>(a < 0 ? 0 : (a > rows ? rows : a));
    }
    return min(max(static_cast<const int32_t*>(cu)[n], 0), rows);
  }
  __device__ __forceinline__ void range(int32_t n, int32_t& a, int32_t& b) const {
    a = start(n);
    b = max(a, start(n + 1));
  }
};

// State slot of sequence n: -1 when it has none (negative, or out of range, which is
// recorded by the thread that `reports`).
__device__ __forceinline__ int32_t state_slot(const int32_t* idx, int32_t n, int32_t pool,
                                              int32_t* status, bool reports) {
  if (idx == nullptr) return n;
  const int32_t i = idx[n];
  if (i >= pool) {
    if (reports && status != nullptr) atomicCAS(status, 0, kStatusBadIndex);
    return -1;
  }
  return max(i, -1);
}

// ---- kernel parameters ---------------------------------------------------------------
struct ConvParams {
  const void* x;
  const float* weight;      // [C][W]
  const float* bias;        // [C] or NULL
  void* state;              // [P][W-1][C] or NULL
  const int32_t* slot;
  const uint8_t* has;
  void* out;                // [parts][rows][C / parts]
  void* steps;              // decode: [N][T][W-1][C] or NULL
  int32_t* status;
  Seqs seq;                 // decode: fixed_len = T
  int64_t x_stride;
  int32_t C, part_c, pool;
  int32_t silu, keep, vec;
  int32_t strips;           // prompts: row strips in all
  int32_t strips_per_cta;   // prompts: adjacent strips one CTA walks
};

struct ScanParams {
  const void *x, *dt, *B, *Cm, *z;
  const float *A_log, *D, *dt_bias;
  float* state;             // [P][D][N] or NULL
  const int32_t* slot;
  const uint8_t* has;
  void* out;
  float* steps;             // decode: [N][T][D][N] or NULL
  int32_t* status;
  Seqs seq;
  int64_t xs, ds, zs, bs, cs;   // row strides
  int32_t channels, size, groups, per_group, tiles_per_group, pool;
  int32_t softplus, keep;
  int32_t vec_bc;               // prompts: vectors of B and C may be moved whole
  int32_t longest_first;        // prompts: CTAs take the sequences by falling length
};

struct NormParams {
  const void *x, *res, *gate;
  const float* weight;
  void *out, *res_out;
  float* scales;
  int64_t xs, rs, ros, gs;      // token strides
  int64_t rows;                 // tokens * heads
  int32_t heads, width, group, groups;
  int32_t out8, sigmoid;
  int32_t step;                 // elements that may be moved at a time: 8, 4 or 1
  float eps, inv_width;
};

}  // namespace layer
}  // namespace kda
