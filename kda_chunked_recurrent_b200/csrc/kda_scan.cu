// kda_scan.cu — the selective state space scan over packed sequences (prompts) and over a
// state pool (single tokens and drafts).
//
// Per channel c and state element n, with A = -exp(A_log) and d the step of the row:
//   h <- exp(d A) h + (d x) B,     y = sum_n C h + D x,     out = y silu(z)
//
// Every state element is a recurrence of its own: one exponential, three products and a sum
// per row, and a sum over the elements of a channel.  With 16 elements a channel and 16-bit
// rows that is 16 exponentials for 8 bytes, and an SM makes 16 exponentials a clock, so
// prompts are bound by the special-function units (about 2.2 TB/s of row bytes), not by HBM;
// single tokens, which move 8 bytes of state per exponential, by HBM.
//
// Prompts.  A CTA takes one sequence and a tile of channels through all its rows, the state
// in registers.  A channel's elements lie on kL lanes, kS a lane, so that one sequence of a
// few thousand channels already fills the SMs.  Four scan warps do nothing but the
// recurrence; four helper warps, one block of kTB rows ahead, load the next rows, form d and
// d x once per (row, channel) and the FP32 rows of B and C in shared memory, and, one block
// behind, turn the sums into output rows (skip, gate, rounding).  One barrier a block.
// The sum over a channel's lanes is done for four rows at a time: two exchange steps leave
// each lane with one row's sum (three shuffles for four rows).
//
// Tokens.  Four state elements (16 bytes) per thread, the state read and written once; a
// CTA takes several sequences so that A stays in registers.
#include <type_traits>

#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace scan {

constexpr int kTB = 32;         // rows per block
constexpr int kHelpers = 128;   // helper threads
constexpr int kU = 4;           // rows per step of the scan

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

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1], with the logarithm from the
// series of the inverse hyperbolic tangent, log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// which is relatively exact for a small e too (a step of 1e-3 is the usual case, and its
// relative error is the state's): the first term left out is s^15 / 15, below 2^-27 of s.
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 e = make_float2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
  const float2 t = add2<true>(e, splat(2.f));
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

// kNP state elements per channel (padded), kS of them per lane, kK channels per lane, kSW scan
// warps; kPoly of the kU kS / 2 pairs of exponentials of a step and channel have one on the
// FMA pipe.
template <typename T, int kNP_, int kS_, int kK_, int kSW_, int kPoly_ = 0>
struct Cfg {
  static constexpr int kNP = kNP_, kS = kS_, kK = kK_, kSW = kSW_, kPoly = kPoly_;
  static constexpr int kL = kNP / kS;                   // lanes per channel
  static constexpr int kCW = 32 / kL;                   // channels side by side in a warp
  static constexpr int kCH = kSW * kCW * kK;            // channels per CTA
  static constexpr int kThreads = 32 * kSW + kHelpers;
  // a helper thread has two rows of kE channels, kParts threads a row, and kQ elements of one
  // row of B and of C
  static constexpr int kE = kCH >= 16 ? kCH / 8 : 2, kParts = kCH / kE, kQ = kNP / 4;
  // row pitch of the sums: a multiple of 4 floats that spreads the four rows which a warp
  // stores together over the banks
  static constexpr int kYP = kCH + (kCH >= 16 ? 8 : 4);
  // 32-bit words of B (as many of C) that a lane reads per row, and of a row of both
  static constexpr int kElem = sizeof(typename T::Raw);
  static constexpr int kLW = kS * 2 * kElem / 4, kRW = kNP * 2 * kElem / 4;
  struct Stage {
    // {d, d} and {d x, d x} of an even row and the next.  Channel part kE + e is at place
    // kParts e + part, here and in the sums: helper threads write, and scan lanes read,
    // adjacent places, and a thread's channels stay adjacent in global memory.
    float4 dd[kTB / 2][kCH];
    // B and C in the rows' own type (half the bytes for 16 bits, and it is the reads from
    // shared memory that bound the scan): per lane q its kS elements of B, then of C
    uint32_t bc[kTB][kRW];
  };
  static __device__ __forceinline__ int channel(int place) {
    return (place % kParts) * kE + place / kParts;
  }
  // Rows on their way: what every helper thread copies for itself, kRing blocks deep (as many
  // as 48 KB hold, at least 4).
  struct Raws {
    typename T::Raw x[2][kHelpers][kE], dt[2][kHelpers][kE], z[2][kHelpers][kE];
    typename T::Raw b[kHelpers][kQ], c[kHelpers][kQ];
  };
  static constexpr int kFit = 48 * 1024 / static_cast<int>(sizeof(Raws));
  static constexpr int kRing = kFit < 4 ? 4 : kFit > 8 ? 8 : kFit;
  struct Smem {
    Raws raw[kRing];
    Stage st[2];
    float y[2][kTB][kYP];
  };
  static_assert(kCH % 8 == 0 && kL >= 4, "helper parts; the exchange of four rows");
};

// 2^y on the FMA pipe: y = n + f, |f| <= 1/2, 2^f = 1 + f P(f) with P of degree 4 fitted for
// the least relative error of 2^f (9e-8 before rounding); n goes into the exponent.  y is
// taken to [-126, 128]: below, the decay is 2^-126; at 128 the result is infinite.
__device__ __forceinline__ float ex2_fma(float y) {
  y = fminf(fmaxf(y, -126.f), 128.f);
  const float big = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer
  const float t = y + big, f = y - (t - big);
  float r = fmaf(f, 0.001326472731307149f, 0.009671512991189957f);
  r = fmaf(f, r, 0.05550733581185341f);
  r = fmaf(f, r, 0.24022242426872253f);
  r = fmaf(f, r, 0.6931470036506653f);
  r = fmaf(f, r, 1.f);
  return __uint_as_float(__float_as_uint(r) + (__float_as_uint(t) << 23));
}

// The operands of kU rows for one lane, read from a stage.
template <typename T, typename C>
struct Rows {
  static constexpr int kP = C::kS / 2 + (C::kS == 1);    // pairs of elements
  uint32_t bc[kU][C::kLW];
  float4 dd[C::kK][kU / 2];
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
      } else if constexpr (C::kLW == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(w);
        bc[u][0] = v.x;
        bc[u][1] = v.y;
      } else {
        bc[u][0] = *w;
      }
    }
#pragma unroll
    for (int k = 0; k < C::kK; ++k)
#pragma unroll
      for (int u = 0; u < kU; u += 2) dd[k][u / 2] = st.dd[(t + u) / 2][ch0 + k * C::kCW];
  }
  // elements 2 i and 2 i + 1 of B (of C), element 0 for kS == 1
  __device__ __forceinline__ float2 pair(int u, int i, bool c) const {
    if constexpr (C::kElem == 4) {
      const uint32_t* w = &bc[u][c ? C::kS : 0];
      return make_float2(__uint_as_float(w[2 * i]), C::kS == 1 ? 0.f : __uint_as_float(w[2 * i + 1]));
    } else if constexpr (C::kS == 1) {
      const float2 v = T::unpack2(bc[u][0]);
      return make_float2(c ? v.y : v.x, 0.f);
    } else {
      return T::unpack2(bc[u][(c ? C::kLW / 2 : 0) + i]);
    }
  }
};

// kU rows of the recurrence: h moves on, sum[k][u] is the lane's part of the read-out.
template <typename T, typename C>
__device__ __forceinline__ void step_rows(const Rows<T, C>& r, float (&h)[C::kK][C::kS],
                                          const float (&A)[C::kK][C::kS], float (&sum)[C::kK][kU]) {
#pragma unroll
  for (int k = 0; k < C::kK; ++k) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float4 dd = r.dd[k][u / 2];
      const float d = u % 2 ? dd.y : dd.x, dx = u % 2 ? dd.w : dd.z;
      if constexpr (C::kS == 1) {
        h[k][0] = fmaf(ex2(d * A[k][0]), h[k][0], dx * r.pair(u, 0, false).x);
        sum[k][u] = r.pair(u, 0, true).x * h[k][0];
      } else {
        float2 acc;
#pragma unroll
        for (int i = 0; i < C::kS; i += 2) {
          const float2 y = mul2<true>(make_float2(d, d), make_float2(A[k][i], A[k][i + 1]));
          const bool fma_pipe = ((u * (C::kS / 2) + i / 2) * C::kPoly) % (kU * C::kS / 2) <
                                                    C::kPoly;
          const float2 a = make_float2(ex2(y.x), fma_pipe ? ex2_fma(y.y) : ex2(y.y));
          const float2 b = mul2<true>(make_float2(dx, dx), r.pair(u, i / 2, false));
          const float2 n = fma2<true>(a, make_float2(h[k][i], h[k][i + 1]), b);
          h[k][i] = n.x;
          h[k][i + 1] = n.y;
          const float2 c = r.pair(u, i / 2, true);
          acc = i == 0 ? mul2<true>(c, n) : fma2<true>(c, n, acc);
        }
        sum[k][u] = acc.x + acc.y;
      }
    }
  }
}

// Sums of kU rows over the kL lanes of a channel: in two exchanges the lanes q, q^1, q^2, q^3
// are left with row q & 3 each, then the other lanes are added.
template <typename C>
__device__ __forceinline__ void reduce_rows(const float (&sum)[C::kK][kU],
                                            float (&yb)[kTB][C::kYP], int t, int ch0, int q) {
  const bool b0 = q & 1, b1 = q & 2;
#pragma unroll
  for (int k = 0; k < C::kK; ++k) {
    const float p0 = (b0 ? sum[k][1] : sum[k][0]) +
                     __shfl_xor_sync(0xffffffffu, b0 ? sum[k][0] : sum[k][1], 1);
    const float p1 = (b0 ? sum[k][3] : sum[k][2]) +
                     __shfl_xor_sync(0xffffffffu, b0 ? sum[k][2] : sum[k][3], 1);
    float v = (b1 ? p1 : p0) + __shfl_xor_sync(0xffffffffu, b1 ? p0 : p1, 2);
#pragma unroll
    for (int o = 4; o < C::kL; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (q < 4) yb[t + q][ch0 + k * C::kCW] = v;
  }
}

// One block's scan by one warp, two groups of kU rows a turn: the next group's operands are
// read while one is worked on, so that a scheduler with a single scan warp is kept busy.
// Rows from nt on have d = 0 and B = C = 0 and change nothing.
template <typename T, typename C>
__device__ __forceinline__ void scan_block(const typename C::Stage& st, float (&yb)[kTB][C::kYP],
                                           float (&h)[C::kK][C::kS], const float (&A)[C::kK][C::kS],
                                           int ch0, int q, int nt) {
  Rows<T, C> r0, r1;
  float s0[C::kK][kU], s1[C::kK][kU];
  r0.load(st, 0, ch0, q);
  for (int t = 0; t < nt; t += 2 * kU) {
    r1.load(st, t + kU, ch0, q);
    step_rows<T, C>(r0, h, A, s0);
    r0.load(st, (t + 2 * kU) % kTB, ch0, q);
    reduce_rows<C>(s0, yb, t, ch0, q);
    step_rows<T, C>(r1, h, A, s1);
    reduce_rows<C>(s1, yb, t + kU, ch0, q);
  }
}

// kVec: the rows' vectors may be moved whole (then a part is inside the tile or outside).
template <typename T, typename C, bool kVec>
__global__ void __launch_bounds__(C::kThreads) kda_scan_prefill_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  constexpr int kE = C::kE, kQ = C::kQ;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  typename C::Smem& sm = *reinterpret_cast<typename C::Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = p.groups * p.tiles_per_group;
  const int32_t n = blockIdx.x / tiles;
  const int tile = blockIdx.x - n * tiles;
  const int grp = tile / p.tiles_per_group;
  const int in_grp = (tile - grp * p.tiles_per_group) * C::kCH;
  const int cbase = grp * p.per_group + in_grp;              // first channel of the tile
  const int nch = min(C::kCH, p.per_group - in_grp);         // channels in it
  int32_t row0, row1;
  p.seq.range(n, row0, row1);
  const int32_t len = row1 - row0, nblk = (len + kTB - 1) / kTB;
  const int32_t slot =
      p.state == nullptr ? -1 : state_slot(p.slot, n, p.pool, p.status, tile == 0 && tid == 0);
  if (len == 0 && slot < 0) return;

  if (warp < C::kSW) {
    // ---- scan warps
    const int q = lane % C::kL, ch0 = warp * (C::kCW * C::kK) + lane / C::kL;   // place
    float h[C::kK][C::kS], A[C::kK][C::kS];
    const bool old = slot >= 0 && (p.has == nullptr || p.has[n] != 0);
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int ch = C::channel(ch0 + k * C::kCW);
#pragma unroll
      for (int i = 0; i < C::kS; ++i) {
        const int e = q * C::kS + i;
        const bool in = ch < nch && e < p.size;
        const int64_t at = static_cast<int64_t>(cbase + ch) * p.size + e;
        // elements past the state's size decay at rate 0 and take nothing: B and C are 0 there
        A[k][i] = in ? -expf(p.A_log[at]) * kLog2e : 0.f;
        h[k][i] = (in && old)
                      ? p.state[static_cast<int64_t>(slot) * p.channels * p.size + at]
                      : 0.f;
      }
    }
    __syncthreads();
    for (int b = 0; b < nblk; ++b) {
      scan_block<T, C>(sm.st[b & 1], sm.y[b & 1], h, A, ch0, q, min(kTB, len - b * kTB));
      __syncthreads();
    }
    if (slot >= 0) {
#pragma unroll
      for (int k = 0; k < C::kK; ++k) {
        const int ch = C::channel(ch0 + k * C::kCW);
#pragma unroll
        for (int i = 0; i < C::kS; ++i) {
          const int e = q * C::kS + i;
          if (ch < nch && e < p.size)
            p.state[(static_cast<int64_t>(slot) * p.channels + cbase + ch) * p.size + e] =
                h[k][i];
        }
      }
    }
    return;
  }

  // ---- helper warps: rows 2 rp and 2 rp + 1 of a block, channels part kE .. + kE - 1; row br
  // of B and C, elements quarter kQ .. + kQ - 1
  const int ht = tid - 32 * C::kSW;
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
  const Raw* X = rows_at(p.x, p.xs, lrow, cbase + cl);
  const Raw* DT = rows_at(p.dt, p.ds, lrow, cbase + cl);
  const Raw* Z = rows_at(p.z, p.zs, lrow, cbase + cl);
  const Raw* Bp = rows_at(p.B, p.bs, brow, static_cast<int64_t>(grp) * p.size + quarter * kQ);
  const Raw* Cp = rows_at(p.Cm, p.cs, brow, static_cast<int64_t>(grp) * p.size + quarter * kQ);
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
  // alignment the elements go through registers.
  const auto bring = [&](auto n_c, Raw* dst, const Raw* src, const void* base, int count) {
    constexpr int kN = decltype(n_c)::value;
    if constexpr (kVec) {
      copy_async<kN * static_cast<int>(sizeof(Raw))>(smem_u32(dst), count > 0 ? src : base,
                                                     count <= 0);
    } else {
      Vec<T, kN> v;
      v.template load<false>(src, count);
      v.template store<true>(dst);
    }
  };
  using NE = std::integral_constant<int, kE>;
  using NQ = std::integral_constant<int, kQ>;
  const auto request = [&](int b) {
    if (b < nblk) {
      typename C::Raws& r = sm.raw[b % C::kRing];
      const int rest = len - b * kTB;      // rows from the block's first on
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int count = 2 * rp + o < rest ? left : 0;
        bring(NE(), r.x[o][ht], X + o * p.xs, p.x, count);
        bring(NE(), r.dt[o][ht], DT + o * p.ds, p.dt, count);
        if (gated) bring(NE(), r.z[o][ht], Z + o * p.zs, p.z, count);
      }
      const int count = br < rest ? left_bc : 0;
      bring(NQ(), r.b[ht], Bp, p.B, count);
      bring(NQ(), r.c[ht], Cp, p.Cm, count);
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
    if constexpr (kHalf == 0) {     // one element of 16 bits each: B low, C high
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = __byte_perm(vb.w[i / 2], vc.w[i / 2], i % 2 ? 0x7632 : 0x5410);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        w[i / kHalf * C::kLW + i % kHalf] = vb.w[i];
        w[i / kHalf * C::kLW + kHalf + i % kHalf] = vc.w[i];
      }
    }
    uint4* to = reinterpret_cast<uint4*>(&st.bc[br][quarter * kWords]);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  };
  const auto finish = [&](int b) {
    const typename C::Raws& raw = sm.raw[b % C::kRing];
    const int rest = len - b * kTB - 2 * rp;
    if (left > 0) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        if (o >= rest) break;
        float xf[kE], zf[kE], y[kE];
        Vec<T, kE> v;
        v.template load<true>(raw.x[o][ht]);
        v.unpack(xf);
#pragma unroll
        for (int e = 0; e < kE; ++e)
          y[e] = fmaf(skip[e], xf[e], sm.y[b & 1][2 * rp + o][C::kParts * e + part]);
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
    if (b > 0) finish(b - 1);
    __syncthreads();
  }
  copy_wait<0>();
  if (nblk > 0) finish(nblk - 1);
}

// ---- tokens: four elements per lane, kL lanes per channel, four sequences at a time.
// A lane's first duty is one of the four sequences: it alone loads dt, x and z there and takes
// the softplus and the gate, and hands them to the other lanes of the channel; and it is left
// with the sum of that sequence after the exchange.
template <typename T, int kL, bool kVec>
__global__ void __launch_bounds__(256, sizeof(typename T::Raw) == 4 ? 2 : 3)
kda_scan_decode_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  constexpr int kCh = 256 / kL;     // channels per CTA
  constexpr int kN = 4;             // sequences per CTA
  const int q = threadIdx.x % kL, cl = threadIdx.x / kL, own = q & 3;
  const int tiles = p.tiles_per_group;                 // channel tiles (groups may share one)
  const int tile = blockIdx.x % tiles;
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / tiles) * kN;
  const int ch = tile * kCh + cl;
  const bool on = ch < p.channels;
  const int c = on ? ch : p.channels - 1;              // idle threads follow the last channel
  const int e0 = 4 * q, count = on ? p.size - e0 : 0;  // state elements of this thread
  const int32_t T_new = p.seq.fixed_len;
  int32_t slot[kN];
#pragma unroll
  for (int s = 0; s < kN; ++s)
    slot[s] = n0 + s < p.seq.num ? state_slot(p.slot, n0 + s, p.pool, p.status,
                                              tile == 0 && threadIdx.x == 0)
                                 : -1;
  const int64_t state_at = static_cast<int64_t>(c) * p.size + e0;
  const int64_t state_slot_size = static_cast<int64_t>(p.channels) * p.size;
  Vec<F32, 4> sv[kN];
#pragma unroll
  for (int s = 0; s < kN; ++s) {
    if (slot[s] >= 0 && count > 0)
      sv[s].template load<kVec>(p.state + slot[s] * state_slot_size + state_at, count);
    else
      sv[s].clear();
  }
  // rows of token 0; token t is t strides on
  const int64_t r_own = static_cast<int64_t>(n0 + own) * T_new;
  const bool own_in = n0 + own < p.seq.num;
  const bool own_live = own_in && (own == 0 ? slot[0] : own == 1 ? slot[1] : own == 2 ? slot[2]
                                                                                      : slot[3]) >= 0;
  const Raw* X = static_cast<const Raw*>(p.x) + r_own * p.xs + c;
  const Raw* DT = static_cast<const Raw*>(p.dt) + r_own * p.ds + c;
  const Raw* Z = static_cast<const Raw*>(p.z) + r_own * p.zs + c;
  Raw* out = static_cast<Raw*>(p.out) + r_own * p.channels + c;
  const int64_t bc_at = static_cast<int64_t>(c / p.per_group) * p.size + e0;
  const Raw* Bp = static_cast<const Raw*>(p.B) + static_cast<int64_t>(n0) * T_new * p.bs + bc_at;
  const Raw* Cp = static_cast<const Raw*>(p.Cm) + static_cast<int64_t>(n0) * T_new * p.cs + bc_at;
  struct Row {
    Raw x, dt, z;
    Vec<T, 4> b[kN], c[kN];
  };
  const auto fetch = [&](Row& r, int32_t t) {
    if (own_live) {
      r.x = X[t * p.xs];
      r.dt = DT[t * p.ds];
      if (p.z != nullptr) r.z = Z[t * p.zs];
    } else {
      r.x = r.dt = r.z = Raw(0);
    }
#pragma unroll
    for (int s = 0; s < kN; ++s) {
      if (slot[s] >= 0 && count > 0) {
        r.b[s].template load<kVec>(Bp + (static_cast<int64_t>(s) * T_new + t) * p.bs, count);
        r.c[s].template load<kVec>(Cp + (static_cast<int64_t>(s) * T_new + t) * p.cs, count);
      } else {
        r.b[s].clear();
        r.c[s].clear();
      }
    }
  };
  Row cur;
  fetch(cur, 0);
  float2 A[2];
  {
    Vec<F32, 4> av;
    if (count > 0) av.template load<kVec>(p.A_log + state_at, count);
    else av.clear();
    float a[4];
    av.unpack(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = i < count ? -expf(a[i]) * kLog2e : 0.f;
    A[0] = make_float2(a[0], a[1]);
    A[1] = make_float2(a[2], a[3]);
  }
  const float bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f;
  const float skip = p.D != nullptr ? p.D[c] : 0.f;
  float2 h[kN][2];
#pragma unroll
  for (int s = 0; s < kN; ++s) {
    h[s][0] = make_float2(__uint_as_float(sv[s].w[0]), __uint_as_float(sv[s].w[1]));
    h[s][1] = make_float2(__uint_as_float(sv[s].w[2]), __uint_as_float(sv[s].w[3]));
  }
  const auto pack_state = [&](int s) {
    sv[s].w[0] = __float_as_uint(h[s][0].x);
    sv[s].w[1] = __float_as_uint(h[s][0].y);
    sv[s].w[2] = __float_as_uint(h[s][1].x);
    sv[s].w[3] = __float_as_uint(h[s][1].y);
  };
  for (int32_t t = 0; t < T_new; ++t) {
    const float x = T::to(cur.x);
    float d = T::to(cur.dt) + bias;
    if (p.softplus) d = softplus(d);
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
        const float2 e = mul2<true>(make_float2(ds, ds), A[i]);
        h[s][i] = fma2<true>(make_float2(ex2(e.x), ex2(e.y)), h[s][i],
                             mul2<true>(make_float2(dxs, dxs),
                                        make_float2(bf[2 * i], bf[2 * i + 1])));
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
    // a padding row's output is zero
    if (on && q < 4 && own_in)
      out[static_cast<int64_t>(t) * p.channels] = T::from(own_live ? y : 0.f);
    if (t + 1 < T_new) fetch(cur, t + 1);
    if (p.steps != nullptr && count > 0) {
#pragma unroll
      for (int s = 0; s < kN; ++s)
        if (slot[s] >= 0) {
          pack_state(s);
          sv[s].template store<kVec>(
              p.steps + (static_cast<int64_t>(n0 + s) * T_new + t) * state_slot_size + state_at,
              count);
        }
    }
  }
  if (!p.keep && count > 0) {
#pragma unroll
    for (int s = 0; s < kN; ++s)
      if (slot[s] >= 0) {
        pack_state(s);
        sv[s].template store<kVec>(p.state + slot[s] * state_slot_size + state_at, count);
      }
  }
}

// ---- host side
// Whether vectors of `bytes` (at most 16 at a time) may be taken from rows of q.
bool whole(const void* q, int64_t stride_bytes, int bytes) {
  const int a = bytes >= 16 ? 16 : bytes;
  return q == nullptr || (reinterpret_cast<uintptr_t>(q) % a == 0 && stride_bytes % a == 0);
}

template <typename T, typename C>
bool go_prefill(ScanParams p, cudaStream_t s) {
  p.tiles_per_group = (p.per_group + C::kCH - 1) / C::kCH;
  constexpr int e = sizeof(typename T::Raw), kRow = C::kE * e, kBc = C::kQ * e;
  const bool vec = whole(p.x, p.xs * e, kRow) && whole(p.dt, p.ds * e, kRow) &&
                   whole(p.z, p.zs * e, kRow) &&
                   whole(p.out, static_cast<int64_t>(p.channels) * e, kRow) &&
                   p.per_group % C::kE == 0 && whole(p.B, p.bs * e, kBc) &&
                   whole(p.Cm, p.cs * e, kBc) && p.size % C::kQ == 0;
  const int64_t grid = static_cast<int64_t>(p.seq.num) * p.groups * p.tiles_per_group;
  if (grid > INT32_MAX) return false;
  constexpr int kSmem = sizeof(typename C::Smem);
  const auto kernel =
      vec ? kda_scan_prefill_kernel<T, C, true> : kda_scan_prefill_kernel<T, C, false>;
  if (kSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
          cudaSuccess)
    return false;
  kernel<<<static_cast<unsigned>(grid), C::kThreads, kSmem, s>>>(p);
  return true;
}

template <typename T>
bool launch_prefill(const ScanParams& p, int sms, cudaStream_t s) {
  if (p.size > 64) return go_prefill<T, Cfg<T, 128, 8, 1, 4>>(p, s);
  if (p.size > 32) return go_prefill<T, Cfg<T, 64, 8, 1, 4>>(p, s);
  if (p.size > 16) return go_prefill<T, Cfg<T, 32, 4, 1, 4>>(p, s);
  const int64_t chains = static_cast<int64_t>(p.seq.num) * p.channels;
  if (chains < 8LL * sms) return go_prefill<T, Cfg<T, 16, 1, 1, 4>>(p, s);
  if (chains < 16LL * sms) return go_prefill<T, Cfg<T, 16, 2, 1, 4>>(p, s);
  if (chains < 64LL * sms) return go_prefill<T, Cfg<T, 16, 4, 1, 4>>(p, s);
  return go_prefill<T, Cfg<T, 16, 4, 2, 4>>(p, s);
}

template <typename T, int kL>
bool go_decode(ScanParams p, cudaStream_t s) {
  constexpr int kCh = 256 / kL, kN = 4, e = sizeof(typename T::Raw);
  p.tiles_per_group = (p.channels + kCh - 1) / kCh;
  const bool vec = p.size % 4 == 0 && whole(p.B, p.bs * e, 4 * e) && whole(p.Cm, p.cs * e, 4 * e) &&
                   whole(p.A_log, 0, 16);
  const int64_t grid = static_cast<int64_t>((p.seq.num + kN - 1) / kN) * p.tiles_per_group;
  if (grid > INT32_MAX) return false;
  const auto kernel = vec ? kda_scan_decode_kernel<T, kL, true> : kda_scan_decode_kernel<T, kL, false>;
  kernel<<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
  return true;
}

template <typename T>
bool launch_decode(const ScanParams& p, cudaStream_t s) {
  if (p.size > 64) return go_decode<T, 32>(p, s);
  if (p.size > 32) return go_decode<T, 16>(p, s);
  if (p.size > 16) return go_decode<T, 8>(p, s);
  return go_decode<T, 4>(p, s);
}

}  // namespace scan

bool launch_scan_prefill(const ScanParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return scan::launch_prefill<Bf16>(p, sms, s);
  if (dtype == 1) return scan::launch_prefill<F16>(p, sms, s);
  return scan::launch_prefill<F32>(p, sms, s);
}
bool launch_scan_decode(const ScanParams& p, int dtype, cudaStream_t s) {
  if (dtype == 0) return scan::launch_decode<Bf16>(p, s);
  if (dtype == 1) return scan::launch_decode<F16>(p, s);
  return scan::launch_decode<F32>(p, s);
}

}  // namespace layer
}  // namespace kda
