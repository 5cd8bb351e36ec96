// kda_conv.cu — the short causal convolution over packed sequences (prompts) and over a
// state pool (single tokens and drafts).
//
//   y[t, c] = act( bias[c] + sum_{j < W} w[c, j] u[t - (W - 1) + j, c] ),   W = 2, 3, 4
//
// Every channel is on its own and every input row is needed by W outputs, so the work is a
// copy with a little arithmetic: 2 bytes in, 2 bytes out, W FMAs and (SiLU) two special
// functions per element.  Bound: HBM, with the special functions not far behind (29K rows of
// 4608 BF16 channels: 81 us of bytes, 58 us of special functions; 102 us measured, 5.2
// TB/s).  That and the figure for tokens are of passes among others, each over inputs that no pass
// just before used; where two forms are compared below, of calls back to back over three sets of
// inputs, which read some 5% less.
//
// Prompts.  A thread owns kV adjacent channels and walks strips of kStrip rows: all rows
// of a strip are loaded at once, a strip ahead (these loads are what keeps HBM busy), the
// W - 1 rows before it are carried over from the strip before or re-read once per CTA.  The
// first W - 1 rows of every sequence need its state instead; they, and the state that the
// sequence leaves, belong to a second set of CTAs, one per (sequence, column block).  Since
// one thread there reads the old state rows of its channels and then writes the new ones,
// and nobody else touches them, the update in place needs no further ordering.
//
// Tokens.  One thread per kV channels of a sequence: state rows and new rows in, outputs
// and the shifted state out (1024 sequences of 4608 BF16 channels 16.9 us, 4.5 TB/s).
#include <algorithm>

#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace conv {

constexpr int kStrip = 6;

// kVec: every row, the weights and the outputs may be read and written 16 bytes at a time
// (then a thread's channels lie in one part); else element by element.
template <bool kVec>
struct Cfg {
  // channels per thread: 8 bytes of a 16-bit row, 16 of FP32 (16 bytes of a 16-bit row took
  // registers that loads in flight need: 157 against 135 us for 29K rows of 4608)
  static constexpr int kV = kVec ? 4 : 1;
};

template <int W, bool kVec>
struct Taps {
  static constexpr int kV = Cfg<kVec>::kV;
  float w[W][kV];      // tap j of the thread's channels
  float bias[kV];

  __device__ __forceinline__ void load(const ConvParams& p, int c0) {
    Vec<F32, kV * W> wv;
    wv.template load<kVec>(p.weight + static_cast<int64_t>(c0) * W);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = __uint_as_float(wv.w[i * W + j]);
      bias[i] = p.bias != nullptr ? p.bias[c0 + i] : 0.f;
    }
  }
  // u: the W window rows, oldest first
  __device__ __forceinline__ void apply(const float (&u)[W][kV], bool act, float (&y)[kV]) const {
    if constexpr (kV == 1) {
      float a = bias[0];
#pragma unroll
      for (int j = 0; j < W; ++j) a = fmaf(w[j][0], u[j][0], a);
      y[0] = act ? a * sigmoid(a) : a;
    } else {
      float2 a[kV / 2];
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) {
        a[i] = make_float2(bias[2 * i], bias[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < W; ++j)
          a[i] = fma2<true>(make_float2(w[j][2 * i], w[j][2 * i + 1]),
                            make_float2(u[j][2 * i], u[j][2 * i + 1]), a[i]);
      }
      if (act) {
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) a[i] = silu2(a[i]);
      }
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) {
        y[2 * i] = a[i].x;
        y[2 * i + 1] = a[i].y;
      }
    }
  }
};

// Where a thread's channels go: parts are contiguous blocks of all rows.
template <typename T, bool kVec>
struct Out {
  static constexpr int kV = Cfg<kVec>::kV;
  using Raw = typename T::Raw;
  Raw* base;   // the thread's first channel of row 0
  int32_t part_c;
  __device__ __forceinline__ Out(const ConvParams& p, int c) : part_c(p.part_c) {
    const int part = c / p.part_c;
    base = static_cast<Raw*>(p.out) + static_cast<int64_t>(part) * p.seq.rows * p.part_c +
           (c - part * p.part_c);
  }
  __device__ __forceinline__ void put(int64_t row, const float (&y)[kV]) const {
    Vec<T, kV> r;
    r.pack(y);
    r.template store<kVec>(base + row * part_c);
  }
};

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

template <typename T, int W, bool kVec>
__device__ __forceinline__ void strips_body(const ConvParams& p, int group, int c0) {
  constexpr int kV = Cfg<kVec>::kV;
  using Raw = typename T::Raw;
  const bool on = c0 < p.C;
  const int32_t rows = p.seq.rows;
  int32_t t0 = group * p.strips_per_cta * kStrip;     // rows < 2^31 - 4096
  const int32_t t_end = min(rows, t0 + p.strips_per_cta * kStrip);
  const int64_t xs = p.x_stride;
  // row t0 - (W - 1) + i is row i of px; it is only looked at where it exists
  const Raw* px = static_cast<const Raw*>(p.x) + (static_cast<int64_t>(t0) - (W - 1)) * xs + c0;
  Vec<T, kV> r[W - 1 + kStrip], next[kStrip];
  // the rows of the strip behind, while this one is worked on
  const auto ahead = [&] {
    const Raw* q = px + (W - 1 + kStrip) * xs;
    if (on && t0 + 2 * kStrip <= rows) {
#pragma unroll
      for (int i = 0; i < kStrip; ++i) next[i].template load<kVec>(q + i * xs);
    } else {
#pragma unroll
      for (int i = 0; i < kStrip; ++i) {
        if (on && t0 + kStrip + i < rows) next[i].template load<kVec>(q + i * xs);
        else next[i].clear();
      }
    }
  };
  if (on && t0 >= W - 1 && t0 + kStrip <= rows) {
#pragma unroll
    for (int i = 0; i < W - 1 + kStrip; ++i) r[i].template load<kVec>(px + i * xs);
  } else {
#pragma unroll
    for (int i = 0; i < W - 1 + kStrip; ++i) {
      const int32_t t = t0 - (W - 1) + i;
      if (on && t >= 0 && t < rows) r[i].template load<kVec>(px + i * xs);
      else r[i].clear();
    }
  }
  Taps<W, kVec> taps;
  if (on) taps.load(p, c0);
  const Out<T, kVec> out(p, on ? c0 : 0);
  int32_t n = find_seq(p.seq, t0), a, b;
  p.seq.range(n, a, b);
  while (true) {
    const bool more = t0 + kStrip < t_end;
    if (more) ahead();
    float u[W][kV];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j].unpack(u[j]);
    const auto row = [&](int i, bool live) {
      r[W - 1 + i].unpack(u[W - 1]);
      if (live) {
        float y[kV];
        taps.apply(u, p.silu, y);
        out.put(t0 + i, y);
      }
#pragma unroll
      for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int v = 0; v < kV; ++v) u[j][v] = u[j + 1][v];
    };
    if (a + W - 1 <= t0 && t0 + kStrip <= b) {
      if (on) {
#pragma unroll
        for (int i = 0; i < kStrip; ++i) row(i, true);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kStrip; ++i) {
        const int32_t t = t0 + i;
        while (t >= b && n + 1 < p.seq.num) p.seq.range(++n, a, b);
        row(i, on && t >= a + (W - 1) && t < b);
      }
    }
    if (!more) break;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = r[kStrip + j];
#pragma unroll
    for (int i = 0; i < kStrip; ++i) r[W - 1 + i] = next[i];
    t0 += kStrip;
    px += kStrip * xs;
  }
}

// The first W - 1 rows of sequence n and the state that it leaves.
template <typename T, int W, bool kVec>
__device__ __forceinline__ void head_body(const ConvParams& p, int32_t n, int c0) {
  constexpr int kV = Cfg<kVec>::kV;
  using Raw = typename T::Raw;
  if (c0 >= p.C) return;
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
    if (old) past[j].template load<kVec>(st + static_cast<int64_t>(j) * p.C);
    else past[j].clear();
    if (j < len) head[j].template load<kVec>(x + static_cast<int64_t>(a + j) * p.x_stride);
    else head[j].clear();
  }
  if (slot >= 0) {
    // row j of the new state is row len + j of [past; inputs]
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int32_t r = len + j;
      if (r >= W - 1) {
        tail[j].template load<kVec>(x + static_cast<int64_t>(a + r - (W - 1)) * p.x_stride);
      } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
          if (k == r) tail[j] = past[k];
      }
    }
  }
  Taps<W, kVec> taps;
  taps.load(p, c0);
  const Out<T, kVec> out(p, c0);
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
      out.put(a + i, y);
    }
  if (slot >= 0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      tail[j].template store<kVec>(st + static_cast<int64_t>(j) * p.C);
  }
}

// Blocks [0, groups * cols) walk strips, blocks behind them take the sequence heads.
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(256)
kda_conv_prefill_kernel(const ConvParams p, int32_t cols, int32_t groups) {
  const int col = blockIdx.x % cols, i = blockIdx.x / cols;
  const int c0 = (col * blockDim.x + threadIdx.x) * Cfg<kVec>::kV;
  if (i < groups) strips_body<T, W, kVec>(p, i, c0);
  else head_body<T, W, kVec>(p, i - groups, c0);
}

// kSeqs sequences at a time, so that their state rows and first new rows are all on their way
// before any is used.  kOne: one new row each and no step states.
template <typename T, int W, bool kVec, int kSeqs, bool kOne>
__global__ void __launch_bounds__(256) kda_conv_decode_kernel(const ConvParams p, int32_t cols) {
  constexpr int kV = Cfg<kVec>::kV;
  using Raw = typename T::Raw;
  const int col = blockIdx.x % cols;
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / cols) * kSeqs;
  const int c0 = (col * blockDim.x + threadIdx.x) * kV;
  if (c0 >= p.C) return;
  const int32_t T_new = kOne ? 1 : p.seq.fixed_len;
  const int64_t row_c = static_cast<int64_t>(p.C);
  int32_t slot[kSeqs];
  Vec<T, kV> win[kSeqs][W];
#pragma unroll
  for (int i = 0; i < kSeqs; ++i)
    slot[i] = n0 + i < p.seq.num ? state_slot(p.slot, n0 + i, p.pool, p.status, c0 == 0) : -1;
  const Raw* x = static_cast<const Raw*>(p.x) + c0;
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const Raw* st = static_cast<const Raw*>(p.state) + slot[i] * ((W - 1) * row_c) + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      if (slot[i] >= 0) win[i][j].template load<kVec>(st + j * row_c);
      else win[i][j].clear();
    if (slot[i] >= 0)
      win[i][W - 1].template load<kVec>(x + static_cast<int64_t>(n0 + i) * T_new * p.x_stride);
    else
      win[i][W - 1].clear();
  }
  Taps<W, kVec> taps;
  taps.load(p, c0);
  const Out<T, kVec> out(p, c0);
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int64_t row0 = static_cast<int64_t>(n0 + i) * T_new;
    if (n0 + i >= p.seq.num) break;
    if (slot[i] < 0) {   // a padding row: zero outputs
      const float zero[kV] = {};
      for (int32_t t = 0; t < T_new; ++t) out.put(row0 + t, zero);
      continue;
    }
    for (int32_t t = 0; t < T_new; ++t) {
      if (t > 0) win[i][W - 1].template load<kVec>(x + (row0 + t) * p.x_stride);
      float u[W][kV], y[kV];
#pragma unroll
      for (int j = 0; j < W; ++j) win[i][j].unpack(u[j]);
      taps.apply(u, p.silu, y);
      out.put(row0 + t, y);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[i][j] = win[i][j + 1];
      if (!kOne && p.steps != nullptr) {
        Raw* sp = static_cast<Raw*>(p.steps) + (row0 + t) * ((W - 1) * row_c) + c0;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[i][j].template store<kVec>(sp + j * row_c);
      }
    }
    if (!p.keep) {
      Raw* st = static_cast<Raw*>(p.state) + slot[i] * ((W - 1) * row_c) + c0;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[i][j].template store<kVec>(st + j * row_c);
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
  const Shape sh = columns(p.C, p.vec ? Cfg<true>::kV : Cfg<false>::kV);
  p.strips = (p.seq.rows + kStrip - 1) / kStrip;
  // Adjacent strips share the weights and the W - 1 rows between them, and the next one's rows
  // are on their way while one is worked on; a CTA walks up to eight while every SM still gets
  // eight CTAs (29K rows of 4608 channels, us: strips of 4 / 6 / 8 rows, eight each, 105 / 96.6 /
  // 100.5; without the next strip's rows, 8 rows, four each, 107.4).
  p.strips_per_cta = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>(8, static_cast<int64_t>(p.strips) * sh.cols / (8LL * sms))));
  const int64_t groups = (p.strips + p.strips_per_cta - 1) / p.strips_per_cta;
  const int64_t grid = (groups + p.seq.num) * sh.cols;
  if (grid > INT32_MAX) return false;
  const auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), sh.threads, 0, s>>>(p, sh.cols,
                                                              static_cast<int32_t>(groups));
  };
  if (W == 2) go(p.vec ? kda_conv_prefill_kernel<T, 2, true> : kda_conv_prefill_kernel<T, 2, false>);
  else if (W == 3) go(p.vec ? kda_conv_prefill_kernel<T, 3, true> : kda_conv_prefill_kernel<T, 3, false>);
  else go(p.vec ? kda_conv_prefill_kernel<T, 4, true> : kda_conv_prefill_kernel<T, 4, false>);
  return true;
}

template <typename T, int W, int kSeqs, bool kOne>
bool go_decode(const ConvParams& p, const Shape& sh, cudaStream_t s) {
  const int64_t grid = static_cast<int64_t>((p.seq.num + kSeqs - 1) / kSeqs) * sh.cols;
  if (grid > INT32_MAX) return false;
  const auto kernel = p.vec ? kda_conv_decode_kernel<T, W, true, kSeqs, kOne>
                            : kda_conv_decode_kernel<T, W, false, kSeqs, kOne>;
  kernel<<<static_cast<unsigned>(grid), sh.threads, 0, s>>>(p, sh.cols);
  return true;
}

template <typename T, int W>
bool pick_decode(const ConvParams& p, int sms, cudaStream_t s) {
  const Shape sh = columns(p.C, p.vec ? Cfg<true>::kV : Cfg<false>::kV);
  const bool one = p.seq.fixed_len == 1 && p.steps == nullptr;
  // Two sequences per thread once the batch fills the SMs without that.
  if (static_cast<int64_t>(p.seq.num) * sh.cols >= 8LL * sms)
    return one ? go_decode<T, W, 2, true>(p, sh, s) : go_decode<T, W, 2, false>(p, sh, s);
  return one ? go_decode<T, W, 1, true>(p, sh, s) : go_decode<T, W, 1, false>(p, sh, s);
}

template <typename T>
bool launch_decode(const ConvParams& p, int W, int sms, cudaStream_t s) {
  if (W == 2) return pick_decode<T, 2>(p, sms, s);
  if (W == 3) return pick_decode<T, 3>(p, sms, s);
  return pick_decode<T, 4>(p, sms, s);
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
