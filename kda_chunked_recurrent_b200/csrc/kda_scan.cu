// kda_scan.cu — the selective state space scan over packed sequences (prompts) and over a
// state pool (single tokens and drafts).
//
// Per channel c and state element n, with A = -exp(A_log) and d the step of the row:
//   h <- exp(d A) h + (d x) B,     y = sum_n C h + D x,     out = y silu(z)
//
// Every state element is a recurrence of its own: one exponential, three products and a sum
// per row, and a sum over the elements of a channel.  With 16 elements a channel and 16-bit
// rows that is 16 exponentials (and 4 more special functions for softplus and gate) for 8
// bytes, and an SM makes 16 a clock, so prompts are bound by the special-function units, at
// about 2 TB/s of row bytes, not by HBM; single tokens, which move 8 bytes of state per
// exponential, by HBM.
//
// Prompts.  A CTA takes one sequence and a tile of channels through all its rows, the state
// in registers.  A channel's elements lie on kL lanes, kS a lane, so that one sequence of a
// few thousand channels already fills the SMs.  Four scan warps do nothing but the
// recurrence.  Four helper warps copy rows into a ring of raw blocks of kTB rows several
// blocks ahead (a row of HBM is about a microsecond away, as long as two blocks take), form d
// and d x once per (row, channel) one block ahead, and, one block behind, add the lanes' parts
// of the sums and write the output rows (skip, gate, rounding).  One barrier a block.
//
// Measured (passes among others, each over inputs that no pass just before used): 8192 rows of
// 4096 BF16 channels 287 us.  At 16 a clock and SM and 1.92 GHz the exponentials alone take 137 on
// the 128 SMs that have work, all special functions, 20 a row and channel, 171 (148 on all 148).  16
// ragged prompts of 2048 FP16 channels 362 us, against 259.  With one scan and one helper warp on a
// scheduler the rest is latency: a row takes 67 clocks, where the scan warp's 4 exponentials a lane
// need 32 and the helpers' special functions 8.  Tried and dropped, us for the first, each beside
// the form of its time: one exponential in eight on the FMA pipe 337 (of 312), B and C in FP32 and d
// in pairs in shared memory 306 (of 285; in pairs alone 294), separate warps for staging and writing
// 283 (of 293), but 386 of 373 for the ragged prompts, two channels per lane 419 (of 401, ragged).
//
// Tokens.  Four state elements (16 bytes) per thread, the state read and written once; four
// sequences at a time.  256 sequences of 4096 channels 33.5 us, 4.3 TB/s.
#include <algorithm>
#include <type_traits>

#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace scan {

constexpr int kTB = 32;         // rows per block
constexpr int kSW = 4;          // scan warps
constexpr int kHelpers = 128;   // helper threads
constexpr int kThreads = 32 * kSW + kHelpers;
constexpr int kU = 2;           // rows per step of the scan

// Asynchronous copy of kBytes (4, 8 or a multiple of 16) from global to shared memory, or of
// as many zeros.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool zero) {
  constexpr int kStep = kBytes >= 16 ? 16 : kBytes;
#pragma unroll
  for (int o = 0; o < kBytes; o += kStep)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst + o),
                 "l"(static_cast<const char*>(src) + o), "n"(kStep), "r"(zero ? 0 : kStep)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// -log2(e) e^v, the decay rate of A_log = v in powers of two.  The rounding of v log2(e) is made
// good: the product's error times ln 2 is added to the exponential relatively, so that a rate is
// off by no more than the exponential's own 2^-22.  Where the product is infinite or far down
// there is no such error to take (infinity less infinity), and near 2^128 the rate leaves FP32
// anyway: it is held at the largest number, so that a step of zero behind it still decays
// nothing.  v = -infinity gives a rate of zero.
__device__ __forceinline__ float decay_rate(float v) {
  const float y = v * kLog2e;
  const float e = fmaf(v, kLog2e, -y) + v * 1.925963033500948e-8f;   // log2(e) - its FP32 value
  float r = ex2(y);
  if (y > -150.f && y < 127.75f) r = fmaf(r, e * 0.6931471805599453f, r);
  return max_nan(-kLog2e * r, -3.402823466e38f);
}

// 2^y h + h0 where 2^y may leave FP32's range though the sum does not: then in three factors,
// held so far out that any number times all three is zero or infinite.  A zero stays zero and an
// infinity infinite, as row by row.
__device__ __forceinline__ float carry(float y, float h, float h0) {
  if (!(fabsf(y) > 126.f)) return fmaf(ex2(y), h, h0);
  const float f = ex2(fminf(fmaxf(y, -378.f), 378.f) * (1.f / 3.f));
  return fmaf(f, f * h * f, h0);
}

// All threads of a cluster: what was written before the arrival is seen after the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
// A float of another CTA of the cluster, at the place of `p` in its shared memory.
__device__ __forceinline__ float cluster_load(const float* p, int rank) {
  float v;
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1], with the logarithm from the
// series of the inverse hyperbolic tangent, log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// which is relatively exact for a small e too (a step of 1e-3 is the usual case, and its
// relative error is the state's): the first term left out is s^15 / 15, below 2^-26 of s.
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 e = make_float2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
  const float2 t = add2<true>(e, splat(2.f));
  // (two reciprocals: the values are of two rows, and one reciprocal of the product would let a
  // later row, a NaN there above all, into an earlier one)
  const float2 s = mul2<true>(e, make_float2(rcp_approx(t.x), rcp_approx(t.y)));
  const float2 q = mul2<true>(s, s);
  float2 r = fma2<true>(q, splat(1.f / 13.f), splat(1.f / 11.f));
  r = fma2<true>(q, r, splat(1.f / 9.f));
  r = fma2<true>(q, r, splat(1.f / 7.f));
  r = fma2<true>(q, r, splat(1.f / 5.f));
  r = fma2<true>(q, r, splat(1.f / 3.f));
  r = fma2<true>(mul2<true>(q, s), r, s);
  return fma2<true>(splat(2.f), r, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v) { return softplus2(make_float2(v, 0.f)).x; }

// kNP state elements per channel (padded), kS of them per lane.
template <typename T, int kNP_, int kS_>
struct Cfg {
  static constexpr int kNP = kNP_, kS = kS_;
  static constexpr int kL = kNP / kS;                   // lanes per channel
  static constexpr int kCW = 32 / kL;                   // channels side by side in a warp
  static constexpr int kCH = kSW * kCW;                 // channels per CTA
  // a helper thread has two rows of kE channels, kParts threads a row, and kQ elements of one
  // row of B and of C
  static constexpr int kE = kCH >= 16 ? kCH / 8 : 2, kParts = kCH / kE, kQ = kNP / 4;
  // the lanes' parts of the sums of a pair of rows, two lanes side by side
  struct Sums {
    float2 part[kTB / 2][kL / 2][kCH][2];
  };
  // 32-bit words of B (as many of C) that a lane reads per row, and of a row of both
  static constexpr int kElem = sizeof(typename T::Raw);
  static constexpr int kLW = kS * 2 * kElem / 4, kRW = kNP * 2 * kElem / 4;
  struct Stage {
    // {d, d} and {d x, d x} of an even row and the next.  Channel part kE + e is at place
    // kParts e + part, here and in the sums: helper threads write, and scan lanes read,
    // adjacent places, and a thread's channels stay adjacent in global memory.
    float4 dd[kTB / 2][kCH];
    // B and C in the rows' own type (half the bytes and one read for 16 bits): per lane q its
    // kS elements of B, then of C
    uint32_t bc[kTB][kRW];
  };
  static __device__ __forceinline__ int channel(int place) {
    return (place % kParts) * kE + place / kParts;
  }
  // Rows on their way: what every helper thread copies for itself, kRing blocks deep (as many
  // as 32 KB hold; at least 4, or 3 of the largest, whose copies then overlap one block only).
  struct Raws {
    typename T::Raw x[2][kHelpers][kE], dt[2][kHelpers][kE], z[2][kHelpers][kE];
    typename T::Raw b[kHelpers][kQ], c[kHelpers][kQ];
  };
  static constexpr int kFit = 32 * 1024 / static_cast<int>(sizeof(Raws));
  static constexpr int kLeast = sizeof(Raws) > 32 * 1024 ? 3 : 4;
  static constexpr int kRing = kFit < kLeast ? kLeast : kFit > 8 ? 8 : kFit;
  struct Smem {
    Raws raw[kRing];
    Stage st[2];
    Sums y[2];     // (16-byte aligned: what precedes is whole vectors)
  };
  static_assert(kCH % 8 == 0 && kL >= 4, "helper parts; pairs of lanes");
};

// The operands of kU rows for one lane, read from a stage.
template <typename T, typename C>
struct Rows {
  uint32_t bc[kU][C::kLW];
  float4 dd[kU / 2];
  __device__ __forceinline__ void load(const typename C::Stage& st, int t, int ch0, int q) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t* w = &st.bc[t + u][q * C::kLW];
      if constexpr (C::kLW % 4 == 0) {
#pragma unroll
        for (int i = 0; i < C::kLW / 4; ++i) {
          const uint4 v = reinterpret_cast<const uint4*>(w)[i];
          bc[u][4 * i] = v.x;
          bc[u][4 * i + 1] = v.y;
          bc[u][4 * i + 2] = v.z;
          bc[u][4 * i + 3] = v.w;
        }
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(w);
        bc[u][0] = v.x;
        bc[u][1] = v.y;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; u += 2) dd[u / 2] = st.dd[(t + u) / 2][ch0];
  }
  // elements 2 i and 2 i + 1 of B (of C)
  __device__ __forceinline__ float2 pair(int u, int i, bool c) const {
    if constexpr (C::kElem == 4) {
      const uint32_t* w = &bc[u][(c ? C::kS : 0) + 2 * i];
      return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    } else {
      return T::unpack2(bc[u][(c ? C::kLW / 2 : 0) + i]);
    }
  }
};

// What a step needs of its rows besides the state: decays, inputs, and C.
template <typename C>
struct Ops {
  static constexpr int kP = C::kS / 2;      // pairs of elements
  float2 a[kU][kP], b[kU][kP], c[kU][kP];
};

// Row u's decays, inputs and C.
template <typename T, typename C>
__device__ __forceinline__ void prepare_row(const Rows<T, C>& r, const float (&A)[C::kS],
                                            Ops<C>& o, int u) {
  const float4 dd = r.dd[u / 2];
  const float d = u % 2 ? dd.y : dd.x, dx = u % 2 ? dd.w : dd.z;
#pragma unroll
  for (int i = 0; i < Ops<C>::kP; ++i) {
    const float2 y = mul2<true>(splat(d), make_float2(A[2 * i], A[2 * i + 1]));
    o.a[u][i] = make_float2(ex2(y.x), ex2(y.y));
    o.b[u][i] = mul2<true>(splat(dx), r.pair(u, i, false));
    o.c[u][i] = r.pair(u, i, true);
  }
}

// Row u of the recurrence: h moves on; the lane's part of the read-out is returned.
template <typename C>
__device__ __forceinline__ float run_row(const Ops<C>& o, float2 (&h)[Ops<C>::kP], int u) {
  float2 acc;
#pragma unroll
  for (int i = 0; i < Ops<C>::kP; ++i) {
    h[i] = fma2<true>(o.a[u][i], h[i], o.b[u][i]);
    acc = i == 0 ? mul2<true>(o.c[u][0], h[0]) : fma2<true>(o.c[u][i], h[i], acc);
  }
  return acc.x + acc.y;
}

// One block's scan by one warp.  A scheduler may have a single scan warp, so its instructions
// are interleaved here: beside the recurrence of one step stand the exponentials of the next
// and the shared-memory reads of the one after.  Rows from nt on have d = 0 and B = C = 0 and
// change nothing.
// kOut false: the state alone, and the sum of the steps d in `d_sum`.
template <typename T, typename C, bool kOut>
__device__ __forceinline__ void scan_block(const typename C::Stage& st, typename C::Sums& y,
                                           float2 (&h)[Ops<C>::kP], const float (&A)[C::kS],
                                           float& d_sum, int ch0, int q, int nt) {
  Rows<T, C> r0, r1;
  Ops<C> o0, o1;
  r0.load(st, 0, ch0, q);
  r1.load(st, kU, ch0, q);
#pragma unroll
  for (int u = 0; u < kU; ++u) prepare_row<T, C>(r0, A, o0, u);
  const auto step = [&](int t, Rows<T, C>& far, const Rows<T, C>& near, Ops<C>& next,
                        const Ops<C>& now) {
    float sum[kU];
    far.load(st, (t + 2 * kU) % kTB, ch0, q);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      prepare_row<T, C>(near, A, next, u);
      sum[u] = run_row<C>(now, h, u);
    }
    // The lane's parts of the sums as they are: the helper that writes the rows adds the kL
    // parts (cheaper than exchanging them between the scan's lanes).
#pragma unroll
    for (int u = 0; u < kU; u += 2) {
      if constexpr (kOut) {
        y.part[(t + u) / 2][q / 2][ch0][q % 2] = make_float2(sum[u], sum[u + 1]);
      } else {
        const float4 dd = st.dd[(t + u) / 2][ch0];
        d_sum += dd.x + dd.y;
      }
    }
  };
  if (nt == kTB && kOut) {
    // A whole block without a branch: what the loop leaves unhidden at its ends was 6% of the
    // time (4096 channels 312 -> 293 us).
#pragma unroll
    for (int t = 0; t < kTB; t += 2 * kU) {
      step(t, r0, r1, o1, o0);
      step(t + kU, r1, r0, o0, o1);
    }
  } else {
#pragma unroll 1
    for (int t = 0; t < nt; t += 2 * kU) {
      step(t, r0, r1, o1, o0);
      step(t + kU, r1, r0, o0, o1);
    }
  }
}

// What the CTAs of a cluster tell one another: per scan lane, the state that its rows leave
// when they start from zeros, and the sum of their steps.
template <typename C>
struct Exchange {
  float h[32 * kSW][C::kS], d[32 * kSW];
};

// kVec: the rows' vectors may be moved whole (then a part is inside the tile or outside).
// kSplit > 1: a cluster of kSplit CTAs shares the rows of one sequence and tile.  Each first
// takes its run of rows from a zero state; over run j a state h becomes
//   exp(A sum_j d) h + h_j,
// so every CTA has the state before its run from its predecessors' h_j and sums, and takes the
// run again with outputs.
template <typename T, typename C, bool kVec, int kSplit>
__global__ void __launch_bounds__(kThreads, 2) kda_scan_prefill_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  constexpr int kE = C::kE, kQ = C::kQ;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  typename C::Smem& sm = *reinterpret_cast<typename C::Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = p.groups * p.tiles_per_group;
  const int seg = blockIdx.x % kSplit, unit = blockIdx.x / kSplit;
  int32_t n = unit / tiles;
  const int tile = unit - n * tiles;
  // Ragged batches that do not run all at once: the longest sequences first, so that the last
  // CTAs to start are short (16 prompts of 1 to 4096 rows: 554 -> 419 us).
  if (p.longest_first) {
    int32_t* lens = reinterpret_cast<int32_t*>(smem_raw);
    int32_t* found = lens + kThreads;
    int32_t mine = 0;
    if (tid < p.seq.num) {
      int32_t a, b;
      p.seq.range(tid, a, b);
      mine = b - a;
      lens[tid] = mine;
    }
    __syncthreads();
    if (tid < p.seq.num) {
      int32_t rank = 0;
      for (int i = 0; i < p.seq.num; ++i) rank += lens[i] > mine || (lens[i] == mine && i < tid);
      if (rank == n) *found = tid;
    }
    __syncthreads();
    n = *found;
    __syncthreads();
  }
  const int grp = tile / p.tiles_per_group;
  const int in_grp = (tile - grp * p.tiles_per_group) * C::kCH;
  const int cbase = grp * p.per_group + in_grp;              // first channel of the tile
  const int nch = min(C::kCH, p.per_group - in_grp);         // channels in it
  int32_t row0, row1;
  p.seq.range(n, row0, row1);
  const int32_t slot = p.state == nullptr ? -1
                                          : state_slot(p.slot, n, p.pool, p.status,
                                                       tile == 0 && seg == 0 && tid == 0);
  bool leaves_state = slot >= 0;
  if constexpr (kSplit > 1) {
    // runs of whole blocks; the CTA of the last row (of the first run, without rows) leaves
    // the state
    const int32_t blocks = (row1 - row0 + kTB - 1) / kTB, per = (blocks + kSplit - 1) / kSplit;
    leaves_state = leaves_state && seg == (blocks == 0 ? 0 : (blocks - 1) / per);
    row0 = min(row0 + seg * per * kTB, row1);
    row1 = min(row0 + per * kTB, row1);
  } else if (row0 == row1 && slot < 0) {
    return;
  }
  const int32_t len = row1 - row0, nblk = (len + kTB - 1) / kTB;
  Exchange<C>& ex = *reinterpret_cast<Exchange<C>*>(smem_raw + sizeof(typename C::Smem));

  if (warp < kSW) {
    // ---- scan warps
    // Adjacent lanes take adjacent channels of one place of the state: a read of B or C is
    // then one address for 8 lanes side by side, one pass of shared memory and not the two that
    // addresses alternating from lane to lane take (293 -> 285 us; state size 64 258 -> 215).
    const int q = lane / C::kCW, ch0 = warp * C::kCW + lane % C::kCW;   // place
    const int ch = C::channel(ch0);
    float2 h[Ops<C>::kP];
    float A[C::kS];
    const bool old = slot >= 0 && (p.has == nullptr || p.has[n] != 0);
    const int64_t at = static_cast<int64_t>(cbase + ch) * p.size + q * C::kS;
    float* state = p.state + static_cast<int64_t>(slot) * p.channels * p.size + at;
#pragma unroll
    for (int i = 0; i < C::kS; ++i) {
      const bool in = ch < nch && q * C::kS + i < p.size;
      // elements past the state's size decay at rate 0 and take nothing: B and C are 0 there
      A[i] = in ? decay_rate(p.A_log[at + i]) : 0.f;
      const float v = (in && old) ? state[i] : 0.f;
      if (i % 2 == 0) h[i / 2].x = v;
      else h[i / 2].y = v;
    }
    const auto run = [&](auto out, float2 (&hh)[Ops<C>::kP], float& d_sum) {
      __syncthreads();
      for (int b = 0; b < nblk; ++b) {
        scan_block<T, C, decltype(out)::value>(sm.st[b & 1], sm.y[b & 1], hh, A, d_sum, ch0, q,
                                               min(kTB, len - b * kTB));
        __syncthreads();
      }
    };
    float d_sum = 0.f;
    if constexpr (kSplit > 1) {
      float2 hl[Ops<C>::kP];
#pragma unroll
      for (int i = 0; i < Ops<C>::kP; ++i) hl[i] = make_float2(0.f, 0.f);
      run(std::false_type(), hl, d_sum);
#pragma unroll
      for (int i = 0; i < C::kS; ++i) ex.h[tid][i] = i % 2 == 0 ? hl[i / 2].x : hl[i / 2].y;
      ex.d[tid] = d_sum;
      cluster_arrive();
      cluster_wait();
      for (int j = 0; j < seg; ++j) {
        const float d = cluster_load(&ex.d[tid], j);
#pragma unroll
        for (int i = 0; i < Ops<C>::kP; ++i) {
          const float2 y = mul2<true>(splat(d), make_float2(A[2 * i], A[2 * i + 1]));
          h[i].x = carry(y.x, h[i].x, cluster_load(&ex.h[tid][2 * i], j));
          h[i].y = carry(y.y, h[i].y, cluster_load(&ex.h[tid][2 * i + 1], j));
        }
      }
      cluster_arrive();     // the neighbours' shared memory is not looked at any more
    }
    run(std::true_type(), h, d_sum);
    if (leaves_state) {
#pragma unroll
      for (int i = 0; i < C::kS; ++i)
        if (ch < nch && q * C::kS + i < p.size) state[i] = i % 2 == 0 ? h[i / 2].x : h[i / 2].y;
    }
    if constexpr (kSplit > 1) cluster_wait();
    return;
  }

  // ---- helper warps: rows 2 rp and 2 rp + 1 of a block, channels part kE .. + kE - 1; row br
  // of B and C, elements quarter kQ .. + kQ - 1
  const int ht = tid - 32 * kSW;
  const int rp = ht / C::kParts, part = ht % C::kParts, br = ht >> 2, quarter = ht & 3;
  const int cl = part * kE;
  const int left = rp < kTB / 2 ? nch - cl : 0;      // channels of this thread in the tile
  const int left_bc = p.size - quarter * kQ;
  const bool gated = p.z != nullptr;
  const auto rows_at = [&](const void* base, int64_t stride, int64_t row, int64_t off) {
    return static_cast<const Raw*>(base) + row * stride + off;
  };
  // rows of the block that is copied next
  const int64_t lrow = static_cast<int64_t>(row0) + 2 * rp, brow = static_cast<int64_t>(row0) + br;
  const Raw *X = nullptr, *DT = nullptr, *Z = nullptr, *Bp = nullptr, *Cp = nullptr;
  // row of the block that is written next
  Raw* O = static_cast<Raw*>(p.out) + lrow * p.channels + cbase + cl;
  float2 bias[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e)
    bias[e] = splat((p.dt_bias != nullptr && e < left) ? p.dt_bias[cbase + cl + e] : 0.f);
  float skip[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e)
    skip[e] = (p.D != nullptr && e < left) ? p.D[cbase + cl + e] : 0.f;

  // Ask for a thread's rows of block b (zeros where there are none).  Without the vectors'
  // alignment the elements come one by one; 16-bit ones, which no asynchronous copy takes, go
  // through registers: all are read, then all are put down.
  const auto request = [&](int b) {
    if (b < nblk) {
      typename C::Raws& r = sm.raw[b % C::kRing];
      const int rest = len - b * kTB;      // rows from the block's first on
      const int n_bc = br < rest ? left_bc : 0;
      int n_row[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) n_row[o] = 2 * rp + o < rest ? left : 0;
      if constexpr (kVec) {
        constexpr int kRow = kE * C::kElem, kBc = kQ * C::kElem;
        const auto bring = [&](auto size, const Raw* dst, const Raw* src, const void* base, int n) {
          copy_async<decltype(size)::value>(smem_u32(dst), n > 0 ? src : base, n <= 0);
        };
        const std::integral_constant<int, kRow> row{};
        const std::integral_constant<int, kBc> bc{};
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          bring(row, r.x[o][ht], X + o * p.xs, p.x, n_row[o]);
          bring(row, r.dt[o][ht], DT + o * p.ds, p.dt, n_row[o]);
          if (gated) bring(row, r.z[o][ht], Z + o * p.zs, p.z, n_row[o]);
        }
        bring(bc, r.b[ht], Bp, p.B, n_bc);
        bring(bc, r.c[ht], Cp, p.Cm, n_bc);
      } else if constexpr (C::kElem == 4) {
        const auto bring = [&](auto size, const Raw* dst, const Raw* src, const void* base, int n) {
#pragma unroll
          for (int i = 0; i < decltype(size)::value; ++i)
            copy_async<4>(smem_u32(dst + i), i < n ? src + i : base, i >= n);
        };
        const std::integral_constant<int, kE> row{};
        const std::integral_constant<int, kQ> bc{};
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          bring(row, r.x[o][ht], X + o * p.xs, p.x, n_row[o]);
          bring(row, r.dt[o][ht], DT + o * p.ds, p.dt, n_row[o]);
          if (gated) bring(row, r.z[o][ht], Z + o * p.zs, p.z, n_row[o]);
        }
        if (p.vec_bc) {
          constexpr int kBc = kQ * C::kElem;
          copy_async<kBc>(smem_u32(r.b[ht]), n_bc > 0 ? Bp : p.B, n_bc <= 0);
          copy_async<kBc>(smem_u32(r.c[ht]), n_bc > 0 ? Cp : p.Cm, n_bc <= 0);
        } else {
          bring(bc, r.b[ht], Bp, p.B, n_bc);
          bring(bc, r.c[ht], Cp, p.Cm, n_bc);
        }
      } else {
        Vec<T, kE> vx[2], vd[2], vz[2];
        Vec<T, kQ> vb, vc;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          vx[o].template load<false>(X + o * p.xs, n_row[o]);
          vd[o].template load<false>(DT + o * p.ds, n_row[o]);
          if (gated) vz[o].template load<false>(Z + o * p.zs, n_row[o]);
        }
        if (p.vec_bc && n_bc > 0) {
          vb.template load<true>(Bp);
          vc.template load<true>(Cp);
        } else {
          vb.template load<false>(Bp, n_bc);
          vc.template load<false>(Cp, n_bc);
        }
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          vx[o].template store<true>(r.x[o][ht]);
          vd[o].template store<true>(r.dt[o][ht]);
          if (gated) vz[o].template store<true>(r.z[o][ht]);
        }
        vb.template store<true>(r.b[ht]);
        vc.template store<true>(r.c[ht]);
      }
      X += kTB * p.xs;
      DT += kTB * p.ds;
      Z += kTB * p.zs;
      Bp += kTB * p.bs;
      Cp += kTB * p.cs;
    }
    copy_commit();
  };
  // rows past the sequence get d = 0: the state stays, their sums are not used
  const auto stage = [&](int b) {
    typename C::Stage& st = sm.st[b & 1];
    const typename C::Raws& raw = sm.raw[b % C::kRing];
    const int rest = len - b * kTB - 2 * rp;
    if (rp < kTB / 2) {
      float x[2][kE], dt[2][kE];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        Vec<T, kE> v;
        v.template load<true>(raw.x[o][ht]);
        v.unpack(x[o]);
        v.template load<true>(raw.dt[o][ht]);
        v.unpack(dt[o]);
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        float2 d = add2<true>(make_float2(dt[0][e], dt[1][e]), bias[e]);
        if (p.softplus) d = softplus2(d);
        if (rest < 2) d = make_float2(rest > 0 ? d.x : 0.f, 0.f);
        const float2 dx = mul2<true>(d, make_float2(x[0][e], x[1][e]));
        st.dd[rp][C::kParts * e + part] = make_float4(d.x, d.y, dx.x, dx.y);
      }
    }
    // the words of kQ elements: kS of B, kS of C, lane by lane
    constexpr int kWords = kQ * 2 * C::kElem / 4, kHalf = C::kLW / 2;
    Vec<T, kQ> vb, vc;
    vb.template load<true>(raw.b[ht]);
    vc.template load<true>(raw.c[ht]);
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords / 2; ++i) {
      w[i / kHalf * C::kLW + i % kHalf] = vb.w[i];
      w[i / kHalf * C::kLW + kHalf + i % kHalf] = vc.w[i];
    }
    uint4* to = reinterpret_cast<uint4*>(&st.bc[br][quarter * kWords]);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  };
  const auto finish = [&](int b) {
    const typename C::Raws& raw = sm.raw[b % C::kRing];
    const int rest = len - b * kTB - 2 * rp;
    if (left > 0 && rest > 0) {
      float2 sum[kE];      // of both rows
#pragma unroll
      for (int e = 0; e < kE; ++e) {
#pragma unroll
        for (int l = 0; l < C::kL / 2; ++l) {
          const float4 v = *reinterpret_cast<const float4*>(
              &sm.y[b & 1].part[rp][l][C::kParts * e + part][0]);
          const float2 w = add2<true>(make_float2(v.x, v.y), make_float2(v.z, v.w));
          sum[e] = l == 0 ? w : add2<true>(sum[e], w);
        }
      }
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        if (o >= rest) break;
        float xf[kE], zf[kE], y[kE];
        Vec<T, kE> v;
        v.template load<true>(raw.x[o][ht]);
        v.unpack(xf);
#pragma unroll
        for (int e = 0; e < kE; ++e) y[e] = fmaf(skip[e], xf[e], o ? sum[e].y : sum[e].x);
        if (gated) {
          v.template load<true>(raw.z[o][ht]);
          v.unpack(zf);
#pragma unroll
          for (int e = 0; e < kE; e += 2) {
            const float2 g = silu2(make_float2(zf[e], zf[e + 1]));
            y[e] *= g.x;
            y[e + 1] *= g.y;
          }
        }
        v.pack(y);
        v.template store<kVec>(O + static_cast<int64_t>(o) * p.channels, left);
      }
    }
    O += static_cast<int64_t>(kTB) * p.channels;
  };

  // Slot b % kRing holds block b from its request to its output, so blocks b - 1 to
  // b + kRing - 2 are there in turn b.  A thread reads back only what it copied itself: its
  // own wait is all the ordering that needs.
  constexpr int kPending = C::kRing - 3;
  const auto run = [&](auto out) {
    constexpr bool kOut = decltype(out)::value;
    X = rows_at(p.x, p.xs, lrow, cbase + cl);
    DT = rows_at(p.dt, p.ds, lrow, cbase + cl);
    Z = rows_at(p.z, p.zs, lrow, cbase + cl);
    Bp = rows_at(p.B, p.bs, brow, static_cast<int64_t>(grp) * p.size + quarter * kQ);
    Cp = rows_at(p.Cm, p.cs, brow, static_cast<int64_t>(grp) * p.size + quarter * kQ);
    for (int b = 0; b < C::kRing - 2; ++b) request(b);
    copy_wait<kPending>();
    if (nblk > 0) stage(0);
    __syncthreads();
    // Turn b, beside the scan of block b: block b + kRing - 2 is asked for, block b + 1 staged,
    // block b - 1 written.
    for (int b = 0; b < nblk; ++b) {
      request(b + C::kRing - 2);
      copy_wait<kPending>();
      if (b + 1 < nblk) stage(b + 1);
      if (kOut && b > 0) finish(b - 1);
      __syncthreads();
    }
    copy_wait<0>();
    if (kOut && nblk > 0) finish(nblk - 1);
  };
  if constexpr (kSplit > 1) {
    run(std::false_type());
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
  }
  run(std::true_type());
  if constexpr (kSplit > 1) cluster_wait();
}

// ---- tokens: four elements per lane, kL lanes per channel, four sequences at a time.
// A lane's first duty is one of the four sequences: it alone loads dt, x and z there and takes
// the softplus and the gate, and hands them to the other lanes of the channel; and it is left
// with the sum of that sequence after the exchange.
enum Tokens {
  kOne,      // one new token each, no step states
  kFew,      // some each, small batches: the next token's rows are loaded a token ahead
  kMany,     // some each, large batches: more warps instead (ahead, the registers of FP32 rows
             // left an SM eight warps: 718 sequences of 7 tokens of 736 channels 135 us)
  kPrompts,  // packed sequences of few rows each
};
template <typename T, int kL, bool kVec, Tokens kMode>
__global__ void __launch_bounds__(256, kMode == kOne    ? (sizeof(typename T::Raw) == 2 ? 4 : 3)
                                       : kMode == kMany ? (sizeof(typename T::Raw) == 2 ? 3 : 2)
                                       : sizeof(typename T::Raw) == 2 ? 2 : 1)
kda_scan_token_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  constexpr int kCh = 256 / kL;     // channels per CTA
  constexpr int kN = 4;             // sequences at a time
  const int q = threadIdx.x % kL, cl = threadIdx.x / kL, own = q & 3;
  const int e0 = 4 * q;                                // first state element of this thread
  const int32_t T_each = kMode == kOne ? 1 : p.seq.fixed_len;   // (not of prompts)
  const int64_t state_slot_size = static_cast<int64_t>(p.channels) * p.size;
  // A unit is a tile of channels of kN sequences; a CTA takes a run of units, whose tiles rarely
  // change (what belongs to the channels is then read again).
  const int32_t batches = (p.seq.num + kN - 1) / kN;
  const int64_t units = static_cast<int64_t>(batches) * p.tiles_per_group;
  const int64_t unit_end = units * (blockIdx.x + 1) / gridDim.x;
  int32_t tile = -1, c = 0, count = 0;
  bool on = false;
  int64_t state_at = 0, bc_at = 0;
  float2 A[2];
  float bias = 0.f, skip = 0.f;

  for (int64_t unit = units * blockIdx.x / gridDim.x; unit < unit_end; ++unit) {
    const int32_t t_of = static_cast<int32_t>(unit / batches);
    const int32_t n0 = static_cast<int32_t>(unit - static_cast<int64_t>(t_of) * batches) * kN;
    if (t_of != tile) {
      tile = t_of;
      const int ch = tile * kCh + cl;
      on = ch < p.channels;
      c = on ? ch : p.channels - 1;                    // idle threads follow the last channel
      count = on ? p.size - e0 : 0;                    // state elements of this thread
      state_at = static_cast<int64_t>(c) * p.size + e0;
      bc_at = static_cast<int64_t>(c / p.per_group) * p.size + e0;
      Vec<F32, 4> av;
      if (count > 0) av.template load<kVec>(p.A_log + state_at, count);
      else av.clear();
      float a[4];
      av.unpack(a);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = i < count ? decay_rate(a[i]) : 0.f;
      A[0] = make_float2(a[0], a[1]);
      A[1] = make_float2(a[2], a[3]);
      bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f;
      skip = p.D != nullptr ? p.D[c] : 0.f;
    }
    int32_t slot[kN];
#pragma unroll
    for (int s = 0; s < kN; ++s)
      slot[s] = n0 + s < p.seq.num && p.state != nullptr
                    ? state_slot(p.slot, n0 + s, p.pool, p.status, tile == 0 && threadIdx.x == 0)
                    : -1;
    // first rows and numbers of rows
    int32_t row[kN], rows[kN], T_new = T_each;
    if constexpr (kMode == kPrompts) T_new = 0;
#pragma unroll
    for (int s = 0; s < kN; ++s) {
      if constexpr (kMode == kPrompts) {
        row[s] = rows[s] = 0;
        if (n0 + s < p.seq.num) {
          int32_t end;
          p.seq.range(n0 + s, row[s], end);
          rows[s] = end - row[s];
        }
        T_new = max(T_new, rows[s]);
      } else {
        row[s] = (n0 + s) * T_each;
        rows[s] = slot[s] >= 0 ? T_each : 0;
      }
    }
    float2 h[kN][2];
    const auto state_of = [&](int s) { return p.state + slot[s] * state_slot_size + state_at; };
#pragma unroll
    for (int s = 0; s < kN; ++s) {
      Vec<F32, 4> v;
      bool old = slot[s] >= 0;
      if constexpr (kMode == kPrompts) old = old && (p.has == nullptr || p.has[n0 + s] != 0);
      if (old && count > 0) v.template load<kVec>(state_of(s), count);
      else v.clear();
      h[s][0] = make_float2(__uint_as_float(v.w[0]), __uint_as_float(v.w[1]));
      h[s][1] = make_float2(__uint_as_float(v.w[2]), __uint_as_float(v.w[3]));
    }
    const auto put_state = [&](int s, float* to) {
      Vec<F32, 4> v;
      v.w[0] = __float_as_uint(h[s][0].x);
      v.w[1] = __float_as_uint(h[s][0].y);
      v.w[2] = __float_as_uint(h[s][1].x);
      v.w[3] = __float_as_uint(h[s][1].y);
      v.template store<kVec>(to, count);
    };
    // the lane's own sequence: rows of token 0; token t is t strides on
    const auto mine = [&](const int32_t (&v)[kN]) {
      return own == 0 ? v[0] : own == 1 ? v[1] : own == 2 ? v[2] : v[3];
    };
    const int32_t rows_own = mine(rows);
    const int64_t r_own = mine(row);
    const Raw* X = static_cast<const Raw*>(p.x) + r_own * p.xs + c;
    const Raw* DT = static_cast<const Raw*>(p.dt) + r_own * p.ds + c;
    const Raw* Z = static_cast<const Raw*>(p.z) + r_own * p.zs + c;
    Raw* out = static_cast<Raw*>(p.out) + r_own * p.channels + c;
    // B and C of the first sequence (prompts: each sequence's rows are found on their own)
    const int64_t b_seq = T_each * p.bs, c_seq = T_each * p.cs;
    const Raw* Bp = static_cast<const Raw*>(p.B) + static_cast<int64_t>(row[0]) * p.bs + bc_at;
    const Raw* Cp = static_cast<const Raw*>(p.Cm) + static_cast<int64_t>(row[0]) * p.cs + bc_at;
    struct Row {
      Raw x, dt, z;
      Vec<T, 4> b[kN], c[kN];
    };
    const auto fetch = [&](Row& r, int32_t t) {       // token t's rows; the pointers move on
      r.x = r.dt = r.z = Raw(0);
      if (t < rows_own) {
        r.x = *X;
        r.dt = *DT;
        if (p.z != nullptr) r.z = *Z;
      }
      const Raw *bs = Bp, *cs = Cp;
#pragma unroll
      for (int s = 0; s < kN; ++s) {
        if constexpr (kMode == kPrompts) {
          bs = static_cast<const Raw*>(p.B) + static_cast<int64_t>(row[s] + t) * p.bs + bc_at;
          cs = static_cast<const Raw*>(p.Cm) + static_cast<int64_t>(row[s] + t) * p.cs + bc_at;
        }
        if (t < rows[s] && count > 0) {
          r.b[s].template load<kVec>(bs, count);
          r.c[s].template load<kVec>(cs, count);
        } else {
          r.b[s].clear();
          r.c[s].clear();
        }
        bs += b_seq;
        cs += c_seq;
      }
      if constexpr (kMode != kOne) {
        X += p.xs;
        DT += p.ds;
        Z += p.zs;
        Bp += p.bs;
        Cp += p.cs;
      }
    };
    constexpr bool kAhead = kMode == kFew || kMode == kPrompts;
    Row cur, next;
    if (kMode != kMany) fetch(cur, 0);
    for (int32_t t = 0; t < T_new; ++t) {
      if (kMode == kMany) fetch(cur, t);
      if (kAhead && t + 1 < T_new) fetch(next, t + 1);
      const float x = T::to(cur.x);
      float d = T::to(cur.dt) + bias;
      if (p.softplus) d = softplus(d);
      if (kMode == kPrompts && t >= rows_own) d = 0.f;     // behind the end: the state stays
      const float dx = d * x;
      float part[kN];
#pragma unroll
      for (int s = 0; s < kN; ++s) {
        // from the lane of this channel whose duty is sequence s
        const int src = (threadIdx.x & 28) | s;
        const float ds = __shfl_sync(0xffffffffu, d, src), dxs = __shfl_sync(0xffffffffu, dx, src);
        float bf[4], cf[4];
        cur.b[s].unpack(bf);
        cur.c[s].unpack(cf);
        float2 acc;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 e = mul2<true>(splat(ds), A[i]);
          h[s][i] = fma2<true>(make_float2(ex2(e.x), ex2(e.y)), h[s][i],
                               mul2<true>(splat(dxs), make_float2(bf[2 * i], bf[2 * i + 1])));
          const float2 cv = make_float2(cf[2 * i], cf[2 * i + 1]);
          acc = i == 0 ? mul2<true>(cv, h[s][0]) : fma2<true>(cv, h[s][1], acc);
        }
        part[s] = acc.x + acc.y;
      }
      // four lanes exchange four sums, each keeps its own; then the other lanes of the channel
      const bool b0 = own & 1, b1 = own & 2;
      const float p0 = (b0 ? part[1] : part[0]) +
                       __shfl_xor_sync(0xffffffffu, b0 ? part[0] : part[1], 1);
      const float p1 = (b0 ? part[3] : part[2]) +
                       __shfl_xor_sync(0xffffffffu, b0 ? part[2] : part[3], 1);
      float y = (b1 ? p1 : p0) + __shfl_xor_sync(0xffffffffu, b1 ? p0 : p1, 2);
#pragma unroll
      for (int o = 4; o < kL; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      y = fmaf(skip, x, y);
      if (p.z != nullptr) {
        const float z = T::to(cur.z);
        y *= z * sigmoid(z);
      }
      // a padding row's output is zero; a prompt has no rows behind its end
      const bool live = t < rows_own;
      if (on && q < 4 && (kMode == kPrompts ? live : n0 + own < p.seq.num))
        *out = T::from(live ? y : 0.f);
      if constexpr (kMode != kOne) {
        out += p.channels;
        if (kAhead) cur = next;
        if (kMode != kPrompts && p.steps != nullptr && count > 0) {
#pragma unroll
          for (int s = 0; s < kN; ++s)
            if (slot[s] >= 0)
              put_state(s, p.steps + (static_cast<int64_t>(row[s] + t) * state_slot_size + state_at));
        }
      }
    }
    if (!p.keep && count > 0) {
#pragma unroll
      for (int s = 0; s < kN; ++s)
        if (slot[s] >= 0) put_state(s, state_of(s));
    }
  }
}

// ---- host side
// Whether vectors of `bytes` (at most 16 at a time) may be taken from rows of q.
bool whole(const void* q, int64_t stride_bytes, int bytes) {
  const int a = bytes >= 16 ? 16 : bytes;
  return q == nullptr || (reinterpret_cast<uintptr_t>(q) % a == 0 && stride_bytes % a == 0);
}

template <typename T, typename C, int kSplit>
bool go_prefill(ScanParams p, int sms, cudaStream_t s) {
  p.tiles_per_group = (p.per_group + C::kCH - 1) / C::kCH;
  constexpr int e = sizeof(typename T::Raw), kRow = C::kE * e, kBc = C::kQ * e;
  p.vec_bc = whole(p.B, p.bs * e, kBc) && whole(p.Cm, p.cs * e, kBc) && p.size % C::kQ == 0;
  const bool vec = whole(p.x, p.xs * e, kRow) && whole(p.dt, p.ds * e, kRow) &&
                   whole(p.z, p.zs * e, kRow) &&
                   whole(p.out, static_cast<int64_t>(p.channels) * e, kRow) &&
                   p.per_group % C::kE == 0 && p.vec_bc;
  const int64_t grid = static_cast<int64_t>(p.seq.num) * p.groups * p.tiles_per_group * kSplit;
  if (grid > INT32_MAX) return false;
  p.longest_first = p.seq.cu != nullptr && p.seq.num > 1 && p.seq.num <= kThreads && grid > sms;
  constexpr int kSmem = sizeof(typename C::Smem) + (kSplit > 1 ? sizeof(Exchange<C>) : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  const auto kernel = vec ? kda_scan_prefill_kernel<T, C, true, kSplit>
                          : kda_scan_prefill_kernel<T, C, false, kSplit>;
  if (kSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
          cudaSuccess)
    return true;        // (CUDA's last error tells)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = kSplit;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = kSplit > 1 ? 1 : 0;
  (void)cudaLaunchKernelEx(&cfg, kernel, p);
  return true;
}

// Few channels and many rows: the rows are shared by a cluster of 8 or 4 CTAs.  A run is taken
// twice, so the time falls to a quarter or a half at best.  Up to 16 elements several CTAs share an
// SM and the clusters may hold twice the SMs; the wider layouts fill an SM's shared memory, and
// clusters that wait for a place cost more than they bring (33 clusters of 4 find one at a time, and
// 9 of 8 or some more).  One sequence, 16-bit rows, us, by one CTA / 4 / 8:
//                              512 rows             4096 rows
//   16 elements,  256 ch   16.6 / 12.5 / 12.5    103 / 53.5 / 43.3
//                 512      16.6 / 12.5 / 12.5    103 / 55.5 / 45.3
//                1024      16.6 / 16.6 / 21.0    104 / 81.4 / 87.0
//   64 elements,  128      33.0 / 24.8 / 24.8    230 /  117 / 71.9
//                 512      33.0 / 25.1 / 45.1    230 /  119 /  136
//                1024      34.6 / 38.9 / 81.7    232 /  236 /  271
//  128 elements,   64      49.4 / 31.0 / 26.6    359 /  174 / 98.5
//                 256      49.3 / 30.9 / 70.3    359 /  175 /  282
//                 512      49.4 / 57.6 /  114    357 /  343 /  469
// and more channels than that fill the SMs without.  FP32 rows turn at the same places.
template <typename T, typename C>
bool pick_prefill(const ScanParams& p, int64_t max_rows, int sms, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>(p.seq.num) * p.groups *
                        ((p.per_group + C::kCH - 1) / C::kCH);
  constexpr bool kWide = C::kNP > 16;
  if (max_rows >= 512) {
    const bool eight = kWide ? tiles * 16 <= sms : tiles * 32 <= 7LL * sms;
    const bool four = kWide ? tiles * 9 <= 2LL * sms : tiles * 4 <= 2LL * sms;
    if (eight) return go_prefill<T, C, 8>(p, sms, s);
    if (four) return go_prefill<T, C, 4>(p, sms, s);
  }
  return go_prefill<T, C, 1>(p, sms, s);
}

template <typename T, int kL>
bool go_tokens(ScanParams p, bool prompts, int sms, cudaStream_t s) {
  constexpr int kCh = 256 / kL, kN = 4, e = sizeof(typename T::Raw);
  p.tiles_per_group = (p.channels + kCh - 1) / kCh;
  const bool vec = p.size % 4 == 0 && whole(p.B, p.bs * e, 4 * e) && whole(p.Cm, p.cs * e, 4 * e) &&
                   whole(p.A_log, 0, 16);
  const bool one = !prompts && p.seq.fixed_len == 1 && p.steps == nullptr;
  const int64_t units =
      static_cast<int64_t>((p.seq.num + kN - 1) / kN) * p.tiles_per_group;
  if (units > INT32_MAX) return false;
  // One token each is short work: as many CTAs as the SMs hold share the units evenly.
  const int64_t grid = one ? std::min<int64_t>(units, sms * (e == 2 ? 4LL : 3LL)) : units;
  const auto go = [&](auto vec_kernel, auto any_kernel) {
    (vec ? vec_kernel : any_kernel)<<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
    return true;
  };
  if (prompts)
    return go(kda_scan_token_kernel<T, kL, true, kPrompts>,
              kda_scan_token_kernel<T, kL, false, kPrompts>);
  if (one)
    return go(kda_scan_token_kernel<T, kL, true, kOne>, kda_scan_token_kernel<T, kL, false, kOne>);
  if (units > 2LL * sms)
    return go(kda_scan_token_kernel<T, kL, true, kMany>,
              kda_scan_token_kernel<T, kL, false, kMany>);
  return go(kda_scan_token_kernel<T, kL, true, kFew>, kda_scan_token_kernel<T, kL, false, kFew>);
}

template <typename T>
bool launch_tokens(const ScanParams& p, bool prompts, int sms, cudaStream_t s) {
  if (p.size > 64) return go_tokens<T, 32>(p, prompts, sms, s);
  if (p.size > 32) return go_tokens<T, 16>(p, prompts, sms, s);
  if (p.size > 16) return go_tokens<T, 8>(p, prompts, sms, s);
  return go_tokens<T, 4>(p, prompts, sms, s);
}

template <typename T>
bool launch_prefill(const ScanParams& p, int64_t max_rows, int sms, cudaStream_t s) {
  // Many sequences of few rows: row by row in the token kernel.  A block of the kernel above costs a
  // CTA about 5 us however few rows it has (above 64 elements, one CTA an SM, 25).  us, token
  // kernel / this one, 16-bit rows:
  //                                        8 rows        16           24           32
  //   16 elements, 32 x 2048 channels   14.6 / 24.8  21.0 / 28.9  28.9 / 31.7  36.6 / 33.3
  //                13 x 2520            13.6 / 14.6  20.7 / 16.6  28.9 / 18.7  35.1 / 19.4
  //                64 x 512             11.3 / 16.6  16.5 / 18.7  22.8 / 19.4  27.1 / 20.7
  //   64 elements, 32 x 2048            41.2 / 66.8  69.6 / 74.0  96.8 / 82.4   130 / 92.5
  //                13 x 2520            29.4 / 33.8  49.2 / 37.4  67.8 / 43.2  86.3 / 47.6
  //  128 elements, 32 x 2048            81.9 /  218   148 /  244   216 /  266   283 /  301
  //                13 x 2520            50.2 /  111  85.8 /  123   120 /  133   155 /  149
  // (at 16 rows of up to 64 elements either may win: even over ten such batches and two types)
  const int64_t ctas = static_cast<int64_t>(p.seq.num) * p.channels / 32;
  if (max_rows <= (p.size > 64 ? 28 : 16) && ctas > 2LL * sms) return launch_tokens<T>(p, true, sms, s);
  if (p.size > 64) return pick_prefill<T, Cfg<T, 128, 8>>(p, max_rows, sms, s);
  if (p.size > 32) return pick_prefill<T, Cfg<T, 64, 8>>(p, max_rows, sms, s);
  if (p.size > 16) return pick_prefill<T, Cfg<T, 32, 4>>(p, max_rows, sms, s);
  // Two elements per lane (16 channels a CTA) while that leaves no SM two CTAs, else four (32
  // channels).  4096 rows of 1024 / 2048 / 2560 channels, us: two 109 / 107 / 167, four 142 /
  // 145 / 145.
  if (static_cast<int64_t>(p.seq.num) * p.channels <= 16LL * sms)
    return pick_prefill<T, Cfg<T, 16, 2>>(p, max_rows, sms, s);
  return go_prefill<T, Cfg<T, 16, 4>, 1>(p, sms, s);
}

}  // namespace scan

bool launch_scan_prefill(const ScanParams& p, int64_t max_rows, int dtype, int sms,
                         cudaStream_t s) {
  if (dtype == 0) return scan::launch_prefill<Bf16>(p, max_rows, sms, s);
  if (dtype == 1) return scan::launch_prefill<F16>(p, max_rows, sms, s);
  return scan::launch_prefill<F32>(p, max_rows, sms, s);
}
bool launch_scan_decode(const ScanParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return scan::launch_tokens<Bf16>(p, false, sms, s);
  if (dtype == 1) return scan::launch_tokens<F16>(p, false, sms, s);
  return scan::launch_tokens<F32>(p, false, sms, s);
}

}  // namespace layer
}  // namespace kda
