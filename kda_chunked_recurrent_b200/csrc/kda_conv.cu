// kda_conv.cu — the short causal convolution over packed sequences (prompts) and over a
// state pool (single tokens and drafts).
//
//   y[t, c] = act( bias[c] + sum_{j < W} w[c, j] u[t - (W - 1) + j, c] ),   W = 2, 3, 4
//
// Every channel is on its own and every input row is needed by W outputs, so the work is a
// copy with a little arithmetic: 2 bytes in, 2 bytes out, W FMAs and (SiLU) two special
// functions per element.  Bound: HBM.
//
// Prompts.  A thread owns kV adjacent channels and walks strips of kStrip rows: all rows
// of a strip are loaded at once (the loads of a strip are what keeps HBM busy), the W - 1
// rows before it are carried over from the strip before or re-read once per CTA.  The
// first W - 1 rows of every sequence need its state instead; they, and the state that the
// sequence leaves, belong to a second set of CTAs, one per (sequence, column block).  Since
// one thread there reads the old state rows of its channels and then writes the new ones,
// and nobody else touches them, the update in place needs no further ordering.
//
// Tokens.  One thread per kV channels of a sequence: state rows and new rows in, outputs
// and the shifted state out.
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace conv {

constexpr int kStrip = 16;

template <typename T>
struct Cfg {
  static constexpr int kV = 4;   // channels per thread: 8 bytes of a 16-bit row, 16 of FP32
};

template <typename T, int W>
struct Taps {
  static constexpr int kV = Cfg<T>::kV;
  float w[kV][W];
  float bias[kV];

  __device__ __forceinline__ void load(const ConvParams& p, int c0) {
    const int n = min(kV, p.C - c0);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[i][j] = i < n ? __ldg(p.weight + static_cast<int64_t>(c0 + i) * W + j) : 0.f;
      bias[i] = (p.bias != nullptr && i < n) ? __ldg(p.bias + c0 + i) : 0.f;
    }
  }
  // u: the W window rows, oldest first
  __device__ __forceinline__ void apply(const float (&u)[W][kV], bool act, float (&y)[kV]) const {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float a = bias[i];
#pragma unroll
      for (int j = 0; j < W; ++j) a = fmaf(w[i][j], u[j][i], a);
      y[i] = act ? silu(a) : a;
    }
  }
};

// Address of out row `row`, channel c0 (parts are contiguous blocks of all rows).
template <typename T>
__device__ __forceinline__ typename T::Raw* out_at(const ConvParams& p, int64_t row, int c) {
  const int part = c / p.part_c;
  return static_cast<typename T::Raw*>(p.out) +
         (static_cast<int64_t>(part) * p.seq.rows + row) * p.part_c + (c - part * p.part_c);
}

// Store kV outputs; without the vector path a thread's channels may straddle two parts.
template <typename T>
__device__ __forceinline__ void put(const ConvParams& p, int64_t row, int c0,
                                    const float (&y)[Cfg<T>::kV]) {
  constexpr int kV = Cfg<T>::kV;
  if (p.vec) {
    Vec<T, kV> r;
    r.pack(y);
    r.store(out_at<T>(p, row, c0), true, kV);
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (c0 + i < p.C) *out_at<T>(p, row, c0 + i) = T::from(y[i]);
  }
}

// The largest n with start(n) <= t, by the whole warp: 32 probes a round.
__device__ __forceinline__ int32_t find_seq(const Seqs& s, int32_t t) {
  if (s.cu == nullptr) return s.fixed_len > 0 ? min(t / s.fixed_len, s.num - 1) : 0;
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = s.num;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int32_t probe = lo + (lane + 1) * step;
    const bool ok = probe < hi && s.start(probe) <= t;
    const int32_t cnt = __popc(__ballot_sync(0xffffffffu, ok));
    hi = min(hi, lo + (cnt + 1) * step);
    lo = min(lo + cnt * step, hi - 1);
  }
  return lo;
}

template <typename T, int W>
__device__ __forceinline__ void strips_body(const ConvParams& p, int group, int c0) {
  constexpr int kV = Cfg<T>::kV;
  using Raw = typename T::Raw;
  const Raw* x = static_cast<const Raw*>(p.x) + c0;
  const bool on = c0 < p.C;
  const int count = p.C - c0;
  const int64_t rows = p.seq.rows;
  int64_t t0 = static_cast<int64_t>(group) * p.strips_per_cta * kStrip;
  const int64_t t_end = min(rows, t0 + static_cast<int64_t>(p.strips_per_cta) * kStrip);
  Vec<T, kV> r[W - 1 + kStrip];
  // row t0 - (W - 1) + i in r[i]
  auto fetch = [&](int from) {
#pragma unroll
    for (int i = 0; i < W - 1 + kStrip; ++i)
      if (i >= from) {
        const int64_t t = t0 - (W - 1) + i;
        if (on && t >= 0 && t < rows) r[i].load(x + t * p.x_stride, p.vec, count);
        else r[i].clear();
      }
  };
  fetch(0);
  Taps<T, W> taps;
  if (on) taps.load(p, c0);
  int32_t n = find_seq(p.seq, static_cast<int32_t>(t0)), a, b;
  p.seq.range(n, a, b);
  while (true) {
    float u[W][kV];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j].unpack(u[j]);
    const bool inside = a + W - 1 <= t0 && t0 + kStrip <= b;
#pragma unroll
    for (int i = 0; i < kStrip; ++i) {
      const int32_t t = static_cast<int32_t>(t0) + i;
      r[W - 1 + i].unpack(u[W - 1]);
      bool live = true;
      if (!inside) {
        while (t >= b && n + 1 < p.seq.num) p.seq.range(++n, a, b);
        live = t >= a + (W - 1) && t < b;
      }
      if (live && on) {
        float y[kV];
        taps.apply(u, p.silu, y);
        put<T>(p, t, c0, y);
      }
#pragma unroll
      for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int v = 0; v < kV; ++v) u[j][v] = u[j + 1][v];
    }
    if (t0 + kStrip >= t_end) break;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = r[kStrip + j];
    t0 += kStrip;
    fetch(W - 1);
  }
}

// The first W - 1 rows of sequence n and the state that it leaves.
template <typename T, int W>
__device__ __forceinline__ void head_body(const ConvParams& p, int32_t n, int c0) {
  constexpr int kV = Cfg<T>::kV;
  using Raw = typename T::Raw;
  if (c0 >= p.C) return;
  const int count = p.C - c0;
  int32_t a, b;
  p.seq.range(n, a, b);
  const int32_t len = b - a;
  const int32_t slot =
      p.state == nullptr ? -1 : state_slot(p.slot, n, p.pool, p.status, c0 == 0);
  if (len == 0 && slot < 0) return;
  const Raw* x = static_cast<const Raw*>(p.x) + c0;
  Raw* st = static_cast<Raw*>(p.state) + static_cast<int64_t>(slot) * (W - 1) * p.C + c0;
  const bool old = slot >= 0 && (p.has == nullptr || p.has[n] != 0);
  Vec<T, kV> past[W - 1], head[W - 1], tail[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (old) past[j].load(st + static_cast<int64_t>(j) * p.C, p.vec, count);
    else past[j].clear();
    if (j < len) head[j].load(x + static_cast<int64_t>(a + j) * p.x_stride, p.vec, count);
    else head[j].clear();
  }
  if (slot >= 0) {
    // row j of the new state is row len + j of [past; inputs]
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int32_t r = len + j;
      if (r >= W - 1) {
        tail[j].load(x + static_cast<int64_t>(a + r - (W - 1)) * p.x_stride, p.vec, count);
      } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
          if (k == r) tail[j] = past[k];
      }
    }
  }
  Taps<T, W> taps;
  taps.load(p, c0);
  float u[2 * (W - 1)][kV];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    past[j].unpack(u[j]);
    head[j].unpack(u[W - 1 + j]);
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i)
    if (i < len) {
      float win[W][kV], y[kV];
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int v = 0; v < kV; ++v) win[j][v] = u[i + j][v];
      taps.apply(win, p.silu, y);
      put<T>(p, a + i, c0, y);
    }
  if (slot >= 0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      tail[j].store(st + static_cast<int64_t>(j) * p.C, p.vec, count);
  }
}

// Blocks [0, groups * cols) walk strips, blocks behind them take the sequence heads.
template <typename T, int W>
__global__ void __launch_bounds__(256)
kda_conv_prefill_kernel(const ConvParams p, int32_t cols, int32_t groups) {
  const int col = blockIdx.x % cols, i = blockIdx.x / cols;
  const int c0 = (col * blockDim.x + threadIdx.x) * Cfg<T>::kV;
  if (i < groups) strips_body<T, W>(p, i, c0);
  else head_body<T, W>(p, i - groups, c0);
}

template <typename T, int W>
__global__ void __launch_bounds__(256) kda_conv_decode_kernel(const ConvParams p, int32_t cols) {
  constexpr int kV = Cfg<T>::kV;
  using Raw = typename T::Raw;
  const int col = blockIdx.x % cols;
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / cols) * p.seqs_per_cta;
  const int c0 = (col * blockDim.x + threadIdx.x) * kV;
  if (c0 >= p.C) return;
  const int count = p.C - c0;
  const int32_t T_new = p.seq.fixed_len, n_end = min(n0 + p.seqs_per_cta, p.seq.num);
  Taps<T, W> taps;
  taps.load(p, c0);
  for (int32_t n = n0; n < n_end; ++n) {
    const int32_t slot = state_slot(p.slot, n, p.pool, p.status, c0 == 0);
    const int64_t row0 = static_cast<int64_t>(n) * T_new;
    if (slot < 0) {   // a padding row: zero outputs
      const float zero[kV] = {};
      for (int32_t t = 0; t < T_new; ++t) put<T>(p, row0 + t, c0, zero);
      continue;
    }
    const Raw* x = static_cast<const Raw*>(p.x) + row0 * p.x_stride + c0;
    Raw* st = static_cast<Raw*>(p.state) + static_cast<int64_t>(slot) * (W - 1) * p.C + c0;
    Vec<T, kV> win[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      win[j].load(st + static_cast<int64_t>(j) * p.C, p.vec, count);
    for (int32_t t = 0; t < T_new; ++t) {
      win[W - 1].load(x + t * p.x_stride, p.vec, count);
      float u[W][kV], y[kV];
#pragma unroll
      for (int j = 0; j < W; ++j) win[j].unpack(u[j]);
      taps.apply(u, p.silu, y);
      put<T>(p, row0 + t, c0, y);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
      if (p.steps != nullptr) {
        Raw* sp = static_cast<Raw*>(p.steps) + (row0 + t) * (W - 1) * p.C + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          win[j].store(sp + static_cast<int64_t>(j) * p.C, p.vec, count);
      }
    }
    if (!p.keep) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        win[j].store(st + static_cast<int64_t>(j) * p.C, p.vec, count);
    }
  }
}

// ---- host side
struct Shape {
  int threads, cols;
};
// A column block of 128 to 256 threads that leaves the fewest threads without channels.
Shape columns(int32_t C, int v) {
  const int units = (C + v - 1) / v;
  Shape best{256, (units + 255) / 256};
  int waste = best.threads * best.cols - units;
  for (int th = 224; th >= 32; th -= 32) {
    const int cols = (units + th - 1) / th;
    if (th < 128 && cols > 1) break;
    if (th * cols - units < waste) {
      waste = th * cols - units;
      best = Shape{th, cols};
    }
  }
  return best;
}

template <typename T>
bool launch_prefill(ConvParams p, int W, int sms, cudaStream_t s) {
  const Shape sh = columns(p.C, Cfg<T>::kV);
  p.strips = (p.seq.rows + kStrip - 1) / kStrip;
  // Adjacent strips share the weights and the W - 1 rows between them; a CTA walks two
  // while that still leaves every SM several CTAs.
  p.strips_per_cta =
      static_cast<int64_t>(p.strips) * sh.cols >= 16LL * sms ? 2 : 1;
  const int64_t groups = (p.strips + p.strips_per_cta - 1) / p.strips_per_cta;
  const int64_t grid = (groups + p.seq.num) * sh.cols;
  if (grid > INT32_MAX) return false;
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), sh.threads, 0, s>>>(p, sh.cols,
                                                              static_cast<int32_t>(groups));
  };
  if (W == 2) go(kda_conv_prefill_kernel<T, 2>);
  else if (W == 3) go(kda_conv_prefill_kernel<T, 3>);
  else go(kda_conv_prefill_kernel<T, 4>);
  return true;
}

template <typename T>
bool launch_decode(ConvParams p, int W, int sms, cudaStream_t s) {
  const Shape sh = columns(p.C, Cfg<T>::kV);
  // Sequences of a CTA share its weights; one CTA takes several once the batch fills the
  // SMs many times over.
  p.seqs_per_cta = static_cast<int64_t>(p.seq.num) * sh.cols >= 32LL * sms ? 4 : 1;
  const int64_t grid = static_cast<int64_t>((p.seq.num + p.seqs_per_cta - 1) / p.seqs_per_cta) *
                       sh.cols;
  if (grid > INT32_MAX) return false;
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), sh.threads, 0, s>>>(p, sh.cols);
  };
  if (W == 2) go(kda_conv_decode_kernel<T, 2>);
  else if (W == 3) go(kda_conv_decode_kernel<T, 3>);
  else go(kda_conv_decode_kernel<T, 4>);
  return true;
}

}  // namespace conv

bool launch_conv_prefill(const ConvParams& p, int W, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return conv::launch_prefill<Bf16>(p, W, sms, s);
  if (dtype == 1) return conv::launch_prefill<F16>(p, W, sms, s);
  return conv::launch_prefill<F32>(p, W, sms, s);
}
bool launch_conv_decode(const ConvParams& p, int W, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return conv::launch_decode<Bf16>(p, W, sms, s);
  if (dtype == 1) return conv::launch_decode<F16>(p, W, sms, s);
  return conv::launch_decode<F32>(p, W, sms, s);
}

}  // namespace layer
}  // namespace kda
