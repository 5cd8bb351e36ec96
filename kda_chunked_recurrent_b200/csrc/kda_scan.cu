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
#include "kda_layer.cuh"

namespace kda {
namespace layer {
namespace scan {

constexpr int kTB = 32;         // rows per block
constexpr int kWarps = 4;       // scan warps; as many helper warps
constexpr int kHelpers = 32 * kWarps;
constexpr int kThreads = 2 * 32 * kWarps;
constexpr int kU = 4;           // rows per step of the scan

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1], with the logarithm from the
// series of the inverse hyperbolic tangent, log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// which is relatively exact for a small e too (a step of 1e-3 is the usual case, and its
// relative error is the state's): the first term left out is s^15 / 15, below 2^-27 of s.
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  const float s = e * rcp_approx(2.f + e), q = s * s;
  float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  r = fmaf(q, r, 1.f / 9.f);
  r = fmaf(q, r, 1.f / 7.f);
  r = fmaf(q, r, 1.f / 5.f);
  r = fmaf(q, r, 1.f / 3.f);
  r = fmaf(q * s, r, s);
  return fmaf(2.f, r, fmaxf(v, 0.f));
}

// kNP state elements per channel (padded), kS of them per lane, kK channels per lane.
template <int kNP_, int kS_, int kK_>
struct Cfg {
  static constexpr int kNP = kNP_, kS = kS_, kK = kK_;
  static constexpr int kL = kNP / kS;                   // lanes per channel
  static constexpr int kCW = 32 / kL;                   // channels side by side in a warp
  static constexpr int kCH = kWarps * kCW * kK;         // channels per CTA
  static constexpr int kE = kCH / 4;                    // channels per helper thread and row
  // row pitch of the sums: a multiple of 4 floats that spreads the four rows which a warp
  // stores together over the banks
  static constexpr int kYP = kCH + (kCH >= 16 ? 8 : 4);
  struct Stage {
    float4 dd[kTB / 2][kCH];          // {d, d x} of an even row, then of the odd row
    float B[kTB][kNP], C[kTB][kNP];
  };
  struct Smem {
    Stage st[2];
    float y[2][kTB][kYP];
  };
};

template <typename T, typename C>
struct Helper {
  using Raw = typename T::Raw;
  static constexpr int kE = C::kE;
  // B and C rows: kNP elements each; four threads a row take a quarter of both
  static constexpr int kQ = C::kNP / 4;
  Vec<T, kE> x[3], z[3];    // blocks in flight: loaded, being scanned, being written
  Vec<T, kE> dt;
  Vec<T, kQ> bq, cq;
};

// One block's scan by one warp.
template <typename C>
__device__ __forceinline__ void scan_block(const typename C::Stage& st, float (&yb)[kTB][C::kYP],
                                           float (&h)[C::kK][C::kS], const float (&A)[C::kK][C::kS],
                                           int ch0, int q, int nt) {
  for (int t = 0; t < nt; t += kU) {
    float sum[C::kK][kU];
    float Bv[kU][C::kS], Cv[kU][C::kS];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if constexpr (C::kS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < C::kS / 4; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(&st.B[t + u][q * C::kS + 4 * i]);
          const float4 c = *reinterpret_cast<const float4*>(&st.C[t + u][q * C::kS + 4 * i]);
          Bv[u][4 * i] = b.x; Bv[u][4 * i + 1] = b.y; Bv[u][4 * i + 2] = b.z; Bv[u][4 * i + 3] = b.w;
          Cv[u][4 * i] = c.x; Cv[u][4 * i + 1] = c.y; Cv[u][4 * i + 2] = c.z; Cv[u][4 * i + 3] = c.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::kS; ++i) {
          Bv[u][i] = st.B[t + u][q * C::kS + i];
          Cv[u][i] = st.C[t + u][q * C::kS + i];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int ch = ch0 + k * C::kCW;
#pragma unroll
      for (int u2 = 0; u2 < kU; u2 += 2) {
        const float4 dd = st.dd[(t + u2) / 2][ch];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int u = u2 + o;
          const float d = o ? dd.z : dd.x, dx = o ? dd.w : dd.y;
          float acc = 0.f;
#pragma unroll
          for (int i = 0; i < C::kS; ++i) {
            const float a = ex2(d * A[k][i]);
            h[k][i] = fmaf(a, h[k][i], dx * Bv[u][i]);
            acc = fmaf(Cv[u][i], h[k][i], acc);
          }
          sum[k][u] = acc;
        }
      }
    }
    // lanes q, q^1, q^2, q^3 exchange so that lane q holds row (q & 3); then the other lanes
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      float v;
      if constexpr (C::kL >= 4) {
        const bool b0 = q & 1, b1 = q & 2;
        const float s0 = b0 ? sum[k][0] : sum[k][1], k0 = b0 ? sum[k][1] : sum[k][0];
        const float s1 = b0 ? sum[k][2] : sum[k][3], k1 = b0 ? sum[k][3] : sum[k][2];
        const float p0 = k0 + __shfl_xor_sync(0xffffffffu, s0, 1);
        const float p1 = k1 + __shfl_xor_sync(0xffffffffu, s1, 1);
        v = (b1 ? p1 : p0) + __shfl_xor_sync(0xffffffffu, b1 ? p0 : p1, 2);
#pragma unroll
        for (int o = 4; o < C::kL; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      }
      if (q < 4) yb[t + q][ch0 + k * C::kCW] = v;
    }
  }
}

template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) kda_scan_prefill_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  static_assert(C::kL >= 4, "the exchange of four rows needs four lanes");
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

  if (warp < kWarps) {
    // ---- scan warps
    const int q = lane % C::kL, ch0 = warp * (C::kCW * C::kK) + lane / C::kL;
    float h[C::kK][C::kS], A[C::kK][C::kS];
    const bool old = slot >= 0 && (p.has == nullptr || p.has[n] != 0);
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int ch = ch0 + k * C::kCW;
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
      scan_block<C>(sm.st[b & 1], sm.y[b & 1], h, A, ch0, q, min(kTB, len - b * kTB));
      __syncthreads();
    }
    if (slot >= 0) {
#pragma unroll
      for (int k = 0; k < C::kK; ++k) {
        const int ch = ch0 + k * C::kCW;
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

  // ---- helper warps: thread -> row ht / 4 of a block, channels (ht % 4) kE .. + kE - 1
  const int ht = tid - kHelpers, r = ht >> 2, part = ht & 3;
  const int cl = part * C::kE, left = nch - cl;      // channels of this thread in the tile
  const Raw* X = static_cast<const Raw*>(p.x) + cbase + cl;
  const Raw* DT = static_cast<const Raw*>(p.dt) + cbase + cl;
  const Raw* Z = static_cast<const Raw*>(p.z) + cbase + cl;
  const Raw* Bp = static_cast<const Raw*>(p.B) + grp * p.size;
  const Raw* Cp = static_cast<const Raw*>(p.Cm) + grp * p.size;
  Raw* O = static_cast<Raw*>(p.out) + cbase + cl;
  const bool gated = p.z != nullptr;
  Helper<T, C> R;
  float bias[C::kE], skip[C::kE];
#pragma unroll
  for (int e = 0; e < C::kE; ++e) {
    bias[e] = (p.dt_bias != nullptr && e < left) ? p.dt_bias[cbase + cl + e] : 0.f;
    skip[e] = (p.D != nullptr && e < left) ? p.D[cbase + cl + e] : 0.f;
  }
  constexpr int kQ = Helper<T, C>::kQ;
  auto load = [&](int b, Vec<T, C::kE>& x, Vec<T, C::kE>& z) {
    const int64_t row = static_cast<int64_t>(row0) + b * kTB + r;
    const bool on = row < row1;
    if (on && left > 0) {
      x.load(X + row * p.xs, p.vec, left);
      R.dt.load(DT + row * p.ds, p.vec, left);
      if (gated) z.load(Z + row * p.zs, p.vec, left);
    } else {
      x.clear();
      R.dt.clear();
    }
    const int n_bc = p.size - part * kQ;
    if (on && n_bc > 0) {
      R.bq.load(Bp + row * p.bs + part * kQ, p.vec_bc, n_bc);
      R.cq.load(Cp + row * p.cs + part * kQ, p.vec_bc, n_bc);
    } else {
      R.bq.clear();
      R.cq.clear();
    }
  };
  // rows past the sequence get d = 0: the state stays, their sums are not used
  auto stage = [&](int b, const Vec<T, C::kE>& x) {
    typename C::Stage& st = sm.st[b & 1];
    const bool on = b * kTB + r < len;
    float xf[C::kE], df[C::kE];
    x.unpack(xf);
    R.dt.unpack(df);
#pragma unroll
    for (int e = 0; e < C::kE; ++e) {
      float d = df[e] + bias[e];
      if (p.softplus) d = softplus(d);
      d = on && e < left ? d : 0.f;
      float2* at = reinterpret_cast<float2*>(&st.dd[r >> 1][cl + e]) + (r & 1);
      *at = make_float2(d, d * xf[e]);
    }
    float f[kQ];
    R.bq.unpack(f);
#pragma unroll
    for (int i = 0; i < kQ; ++i) st.B[r][part * kQ + i] = f[i];
    R.cq.unpack(f);
#pragma unroll
    for (int i = 0; i < kQ; ++i) st.C[r][part * kQ + i] = f[i];
  };
  auto finish = [&](int b, const Vec<T, C::kE>& x, const Vec<T, C::kE>& z) {
    const int64_t row = static_cast<int64_t>(row0) + b * kTB + r;
    if (row >= row1 || left <= 0) return;
    float xf[C::kE], y[C::kE];
    x.unpack(xf);
#pragma unroll
    for (int e = 0; e < C::kE; ++e) y[e] = fmaf(skip[e], xf[e], sm.y[b & 1][r][cl + e]);
    if (gated) {
      float zf[C::kE];
      z.unpack(zf);
#pragma unroll
      for (int e = 0; e < C::kE; ++e) y[e] *= silu(zf[e]);
    }
    Vec<T, C::kE> o;
    o.pack(y);
    o.store(O + row * p.channels, p.vec, left);
  };

  if (nblk > 0) {
    load(0, R.x[0], R.z[0]);
    stage(0, R.x[0]);
    if (nblk > 1) load(1, R.x[1], R.z[1]);
  }
  __syncthreads();
  // before block b: stage b is ready, x[0], z[0] hold block b, x[1], z[1] block b + 1 (in
  // flight), x[2], z[2] block b - 1
  for (int b = 0; b < nblk; ++b) {
    if (b > 0) finish(b - 1, R.x[2], R.z[2]);
    if (b + 1 < nblk) stage(b + 1, R.x[1]);
    R.x[2] = R.x[0];
    R.z[2] = R.z[0];
    R.x[0] = R.x[1];
    R.z[0] = R.z[1];
    if (b + 2 < nblk) load(b + 2, R.x[1], R.z[1]);
    __syncthreads();
  }
  if (nblk > 0) finish(nblk - 1, R.x[2], R.z[2]);
}

// ---- tokens: four elements per lane, kL lanes per channel
template <typename T, int kL>
__global__ void __launch_bounds__(256) kda_scan_decode_kernel(const ScanParams p) {
  using Raw = typename T::Raw;
  constexpr int kCh = 256 / kL;     // channels per CTA
  const int q = threadIdx.x % kL, cl = threadIdx.x / kL;
  const int tiles = p.tiles_per_group;                 // channel tiles (groups may share one)
  const int tile = blockIdx.x % tiles;
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / tiles) * p.seqs_per_cta;
  const int32_t n1 = min(n0 + p.seqs_per_cta, p.seq.num);
  const int ch = tile * kCh + cl;
  const bool on = ch < p.channels;
  const int c = on ? ch : p.channels - 1;              // idle threads follow the last channel
  const int e0 = 4 * q, count = on ? p.size - e0 : 0;  // state elements of this thread
  const int grp = c / p.per_group;
  float A[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    A[i] = i < count ? -expf(p.A_log[static_cast<int64_t>(c) * p.size + e0 + i]) * kLog2e : 0.f;
  const float bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f;
  const float skip = p.D != nullptr ? p.D[c] : 0.f;
  const bool vec_state = p.size % 4 == 0;
  const int32_t T_new = p.seq.fixed_len;
  for (int32_t n = n0; n < n1; ++n) {
    const int32_t slot =
        state_slot(p.slot, n, p.pool, p.status, tile == 0 && threadIdx.x == 0);
    const int64_t r0 = static_cast<int64_t>(n) * T_new;
    Raw* out = static_cast<Raw*>(p.out) + r0 * p.channels + c;
    if (slot < 0) {   // a padding row: zero outputs
      if (on && q == 0)
        for (int32_t t = 0; t < T_new; ++t) out[static_cast<int64_t>(t) * p.channels] = T::from(0.f);
      continue;
    }
    float* st = p.state + (static_cast<int64_t>(slot) * p.channels + c) * p.size + e0;
    Vec<F32, 4> sv;
    if (count > 0) sv.load(st, vec_state, count);
    else sv.clear();
    float h[4];
    sv.unpack(h);
    for (int32_t t = 0; t < T_new; ++t) {
      const int64_t row = r0 + t;
      const float x = T::to(static_cast<const Raw*>(p.x)[row * p.xs + c]);
      float d = T::to(static_cast<const Raw*>(p.dt)[row * p.ds + c]) + bias;
      const float z = p.z != nullptr ? T::to(static_cast<const Raw*>(p.z)[row * p.zs + c]) : 0.f;
      Vec<T, 4> bv, cv;
      if (count > 0) {
        const int64_t at = static_cast<int64_t>(grp) * p.size + e0;
        bv.load(static_cast<const Raw*>(p.B) + row * p.bs + at, p.vec_bc, count);
        cv.load(static_cast<const Raw*>(p.Cm) + row * p.cs + at, p.vec_bc, count);
      } else {
        bv.clear();
        cv.clear();
      }
      if (p.softplus) d = softplus(d);
      const float dx = d * x;
      float bf[4], cf[4], y = 0.f;
      bv.unpack(bf);
      cv.unpack(cf);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(ex2(d * A[i]), h[i], dx * bf[i]);
        y = fmaf(cf[i], h[i], y);
      }
#pragma unroll
      for (int o = 1; o < kL; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      y = fmaf(skip, x, y);
      if (p.z != nullptr) y *= silu(z);
      if (on && q == 0) out[static_cast<int64_t>(t) * p.channels] = T::from(y);
      if (p.steps != nullptr && count > 0) {
        sv.pack(h);
        sv.store(p.steps + (row * p.channels + c) * p.size + e0, vec_state, count);
      }
    }
    if (!p.keep && count > 0) {
      sv.pack(h);
      sv.store(st, vec_state, count);
    }
  }
}

// ---- host side
template <typename T, typename C>
bool go_prefill(ScanParams p, cudaStream_t s) {
  p.tiles_per_group = (p.per_group + C::kCH - 1) / C::kCH;
  constexpr int kBytes = C::kE * static_cast<int>(sizeof(typename T::Raw));
  constexpr int kAlign = kBytes >= 16 ? 16 : kBytes;
  constexpr int kBcBytes = C::kNP / 4 * static_cast<int>(sizeof(typename T::Raw));
  constexpr int kBcAlign = kBcBytes >= 16 ? 16 : kBcBytes;
  const auto ok = [](const void* q, int64_t stride, int align) {
    return q == nullptr || (reinterpret_cast<uintptr_t>(q) % align == 0 &&
                            stride * static_cast<int64_t>(sizeof(typename T::Raw)) % align == 0);
  };
  p.vec = ok(p.x, p.xs, kAlign) && ok(p.dt, p.ds, kAlign) && ok(p.z, p.zs, kAlign) &&
          ok(p.out, p.channels, kAlign) && ok(nullptr, 0, 1) &&
          (p.groups == 1 ||
           p.per_group * static_cast<int64_t>(sizeof(typename T::Raw)) % kAlign == 0);
  p.vec_bc = ok(p.B, p.bs, kBcAlign) && ok(p.Cm, p.cs, kBcAlign) &&
             (p.groups == 1 ||
              p.size * static_cast<int64_t>(sizeof(typename T::Raw)) % kBcAlign == 0);
  const int64_t grid = static_cast<int64_t>(p.seq.num) * p.groups * p.tiles_per_group;
  if (grid > INT32_MAX) return false;
  constexpr int kSmem = sizeof(typename C::Smem);
  auto* kernel = kda_scan_prefill_kernel<T, C>;
  if (kSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
          cudaSuccess)
    return false;
  kernel<<<static_cast<unsigned>(grid), kThreads, kSmem, s>>>(p);
  return true;
}

template <typename T>
bool launch_prefill(const ScanParams& p, int sms, cudaStream_t s) {
  if (p.size > 64) return go_prefill<T, Cfg<128, 8, 1>>(p, s);
  if (p.size > 32) return go_prefill<T, Cfg<64, 8, 1>>(p, s);
  if (p.size > 16) return go_prefill<T, Cfg<32, 4, 1>>(p, s);
  const int64_t chains = static_cast<int64_t>(p.seq.num) * p.channels;
  if (chains < 8LL * sms) return go_prefill<T, Cfg<16, 1, 1>>(p, s);
  if (chains < 16LL * sms) return go_prefill<T, Cfg<16, 2, 1>>(p, s);
  if (chains < 64LL * sms) return go_prefill<T, Cfg<16, 4, 1>>(p, s);
  return go_prefill<T, Cfg<16, 4, 2>>(p, s);
}

template <typename T, int kL>
bool go_decode(ScanParams p, int sms, cudaStream_t s) {
  constexpr int kCh = 256 / kL;
  p.tiles_per_group = (p.channels + kCh - 1) / kCh;
  const auto ok = [](const void* q, int64_t stride) {
    constexpr int a = 4 * static_cast<int>(sizeof(typename T::Raw));
    return reinterpret_cast<uintptr_t>(q) % a == 0 && stride % 4 == 0;
  };
  p.vec_bc = ok(p.B, p.bs) && ok(p.Cm, p.cs) && (p.groups == 1 || p.size % 4 == 0);
  p.seqs_per_cta = static_cast<int64_t>(p.seq.num) * p.tiles_per_group >= 32LL * sms ? 4 : 1;
  const int64_t grid =
      static_cast<int64_t>((p.seq.num + p.seqs_per_cta - 1) / p.seqs_per_cta) * p.tiles_per_group;
  if (grid > INT32_MAX) return false;
  kda_scan_decode_kernel<T, kL><<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
  return true;
}

template <typename T>
bool launch_decode(const ScanParams& p, int sms, cudaStream_t s) {
  if (p.size > 64) return go_decode<T, 32>(p, sms, s);
  if (p.size > 32) return go_decode<T, 16>(p, sms, s);
  if (p.size > 16) return go_decode<T, 8>(p, sms, s);
  return go_decode<T, 4>(p, sms, s);
}

}  // namespace scan

bool launch_scan_prefill(const ScanParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return scan::launch_prefill<Bf16>(p, sms, s);
  if (dtype == 1) return scan::launch_prefill<F16>(p, sms, s);
  return scan::launch_prefill<F32>(p, sms, s);
}
bool launch_scan_decode(const ScanParams& p, int dtype, int sms, cudaStream_t s) {
  if (dtype == 0) return scan::launch_decode<Bf16>(p, sms, s);
  if (dtype == 1) return scan::launch_decode<F16>(p, sms, s);
  return scan::launch_decode<F32>(p, sms, s);
}

}  // namespace layer
}  // namespace kda
