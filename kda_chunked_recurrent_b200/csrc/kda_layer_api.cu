// kda_layer_api.cu — host side of the C ABI declared in include/kda_layer.h: argument
// checks before any launch, then one launch per call on the caller's stream.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <initializer_list>

#include "../../include/kda_layer.h"
#include "kda_layer.cuh"

namespace kda {
namespace layer {
// false: more thread blocks than a launch may have (an error of the launch is CUDA's last error)
bool launch_conv_prefill(const ConvParams& p, int W, int dtype, int sms, cudaStream_t s);
bool launch_conv_decode(const ConvParams& p, int W, int dtype, int sms, cudaStream_t s);
bool launch_scan_prefill(const ScanParams& p, int64_t max_rows, int dtype, int sms,
                         cudaStream_t s);
bool launch_scan_decode(const ScanParams& p, int dtype, int sms, cudaStream_t s);
bool launch_norm(const NormParams& p, int dtype, cudaStream_t s);
}  // namespace layer
}  // namespace kda

using namespace kda::layer;

namespace {

struct Range {
  uintptr_t lo, hi;   // [lo, hi); empty when the pointer is NULL
};
Range rng(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, p == nullptr ? a : a + static_cast<uintptr_t>(bytes)};
}
// bytes from the first to the last element of `rows` rows of `n` elements, `stride` apart
int64_t span(int64_t rows, int64_t stride, int64_t n, int elem) {
  return rows <= 0 ? 0 : ((rows - 1) * stride + n) * elem;
}
bool overlap(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}
bool overlap(const Range& a, std::initializer_list<Range> rs) {
  for (const Range& r : rs)
    if (overlap(a, r)) return true;
  return false;
}
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The kernels count rows, sequences, heads and the elements of a token in 32 bits, and may look a
// block's worth past the last before they find that it is not there.
constexpr int64_t kMost = INT32_MAX - 4096;

int elem_size(int dtype) { return dtype == KDA_DTYPE_F32 ? 4 : 2; }
bool activation_type(int dtype) { return dtype >= KDA_DTYPE_BF16 && dtype <= KDA_DTYPE_F32; }
// 16-byte rows: the fast path of the row kernels
bool rows16(const void* p, int64_t stride, int elem) {
  return p == nullptr || (aligned(p, 16) && stride * elem % 16 == 0);
}

// The current device: capability 10.0 and its SM count.
kda_status_t device(int* sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KDA_ERR_UNSUPPORTED_DEVICE;
  return major == 10 && minor == 0 ? KDA_OK : KDA_ERR_UNSUPPORTED_DEVICE;
}

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// f launches and says whether the work fits one launch; where it does not, nothing was enqueued.
template <typename F>
kda_status_t launch(const char* name, F&& f) {
  NvtxRange nr(name);
  (void)cudaGetLastError();
  const bool fits = f();
  if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH_FAILED;
  return fits ? KDA_OK : KDA_ERR_BAD_SHAPE;
}

// Sequence arguments that conv and scan share.  Decode calls (cu = NULL, per_seq rows each)
// pass rows = num_seqs * per_seq.
struct SeqArgs {
  const int32_t* slot;
  const uint8_t* has;
  const void* cu;
  const int32_t* status;
  bool cu64;
};
kda_status_t check_seqs(const SeqArgs& a, int64_t num, int64_t rows, int64_t pool, bool state,
                        bool decode) {
  if (num < 1 || rows < 0 || num > kMost || rows > kMost) return KDA_ERR_BAD_SHAPE;
  if (a.cu64 && a.cu == nullptr) return KDA_ERR_BAD_OPTION;
  if (!decode && a.cu == nullptr && rows % num != 0) return KDA_ERR_BAD_SHAPE;
  if (state && (pool < 1 || (a.slot == nullptr && pool < num))) return KDA_ERR_BAD_SHAPE;
  if (!state && (a.slot != nullptr || a.has != nullptr)) return KDA_ERR_NULL_ARG;
  if (!aligned(a.slot, 4) || !aligned(a.cu, a.cu64 ? 8 : 4) || !aligned(a.status, 4))
    return KDA_ERR_MISALIGNED;
  return KDA_OK;
}
Seqs make_seqs(const SeqArgs& a, int64_t num, int64_t rows) {
  Seqs s{};
  s.cu = a.cu;
  s.cu64 = a.cu64;
  s.num = static_cast<int32_t>(num);
  s.rows = static_cast<int32_t>(rows);
  s.fixed_len = a.cu == nullptr ? static_cast<int32_t>(rows / num) : 0;
  return s;
}

kda_status_t conv_call(const void* x, const float* weight, const float* bias, void* state,
                       const SeqArgs& sa, const kda_conv_shape_t* sh, void* out, void* steps,
                       int32_t* status, uint32_t flags, bool decode, void* stream) {
  if (sh == nullptr) return KDA_ERR_NULL_ARG;
  const uint32_t known = KDA_CONV_SILU | (decode ? KDA_LAYER_KEEP_STATE : KDA_LAYER_CU_SEQLENS_I64);
  if ((flags & ~known) || sh->reserved != 0 || !activation_type(sh->dtype))
    return KDA_ERR_BAD_OPTION;
  const int64_t N = sh->num_seqs, C = sh->channels, W = sh->width, P = sh->pool_size;
  const int64_t rows = decode ? N * sh->tokens : sh->tokens;
  if (C < 1 || W < 2 || W > 4 || sh->parts < 1 || C % sh->parts != 0 || sh->x_stride < C ||
      (decode && sh->tokens < 1))
    return KDA_ERR_BAD_SHAPE;
  if (C > (1 << 24) || sh->x_stride > (int64_t(1) << 40)) return KDA_ERR_BAD_SHAPE;
  const bool has_state = state != nullptr;
  if (decode && !has_state) return KDA_ERR_NULL_ARG;
  kda_status_t st = check_seqs(sa, N, rows, P, has_state, decode);
  if (st != KDA_OK) return st;
  if (weight == nullptr || (rows > 0 && (x == nullptr || out == nullptr))) return KDA_ERR_NULL_ARG;
  const int e = elem_size(sh->dtype);
  if (!aligned(x, e) || !aligned(state, e) || !aligned(out, e) || !aligned(steps, e) ||
      !aligned(weight, 4) || !aligned(bias, 4))
    return KDA_ERR_MISALIGNED;
  const Range rx = rng(x, span(rows, sh->x_stride, C, e)), rw = rng(weight, C * W * 4),
              rb = rng(bias, C * 4), rst = rng(state, P * (W - 1) * C * e),
              ri = rng(sa.slot, N * 4), rh = rng(sa.has, N),
              rc = rng(sa.cu, (N + 1) * (sa.cu64 ? 8 : 4)), ro = rng(out, rows * C * e),
              rp = rng(steps, rows * (W - 1) * C * e), rs = rng(status, 4);
  for (const Range& o : {ro, rst, rp, rs})
    if (overlap(o, {rx, rw, rb, ri, rh, rc})) return KDA_ERR_OUT_ALIAS;
  if (overlap(ro, {rst, rp, rs}) || overlap(rst, {rp, rs}) || overlap(rp, rs))
    return KDA_ERR_OUT_ALIAS;
  int sms = 0;
  st = device(&sms);
  if (st != KDA_OK) return st;

  ConvParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.state = state;
  p.slot = sa.slot;
  p.has = sa.has;
  p.out = out;
  p.steps = steps;
  p.status = status;
  p.seq = make_seqs(sa, N, rows);
  p.x_stride = sh->x_stride;
  p.C = static_cast<int32_t>(C);
  p.part_c = static_cast<int32_t>(C / sh->parts);
  p.pool = static_cast<int32_t>(P);
  p.silu = (flags & KDA_CONV_SILU) != 0;
  p.keep = (flags & KDA_LAYER_KEEP_STATE) != 0;
  p.vec = rows16(x, sh->x_stride, e) && rows16(state, C, e) && rows16(steps, C, e) &&
          rows16(out, p.part_c, e) && C * e % 16 == 0 && aligned(weight, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch(decode ? "kda_conv_decode" : "kda_conv_prefill", [&] {
    return decode ? launch_conv_decode(p, static_cast<int>(W), sh->dtype, sms, s)
                  : launch_conv_prefill(p, static_cast<int>(W), sh->dtype, sms, s);
  });
}

kda_status_t scan_call(const void* x, const void* dt, const float* A_log, const void* B,
                       const void* C, const float* D, const void* z, const float* dt_bias,
                       float* state, const SeqArgs& sa, const kda_scan_shape_t* sh, void* out,
                       float* steps, int32_t* status, uint32_t flags, bool decode, void* stream) {
  if (sh == nullptr) return KDA_ERR_NULL_ARG;
  const uint32_t known =
      KDA_SCAN_SOFTPLUS | (decode ? KDA_LAYER_KEEP_STATE : KDA_LAYER_CU_SEQLENS_I64);
  if ((flags & ~known) || !activation_type(sh->dtype)) return KDA_ERR_BAD_OPTION;
  const int64_t N = sh->num_seqs, Ch = sh->channels, S = sh->state_size, G = sh->groups,
                P = sh->pool_size;
  const int64_t rows = decode ? N * sh->tokens : sh->tokens;
  if (Ch < 1 || S < 1 || S > 128 || G < 1 || Ch % G != 0 || (decode && sh->tokens < 1) ||
      sh->max_seqlen < 0)
    return KDA_ERR_BAD_SHAPE;
  if (Ch > (1 << 24)) return KDA_ERR_BAD_SHAPE;
  const int64_t most = int64_t(1) << 40;
  if (sh->x_stride < Ch || sh->dt_stride < Ch || (z != nullptr && sh->z_stride < Ch) ||
      sh->b_stride < G * S || sh->c_stride < G * S || sh->x_stride > most ||
      sh->dt_stride > most || (z != nullptr && sh->z_stride > most) || sh->b_stride > most ||
      sh->c_stride > most)
    return KDA_ERR_BAD_SHAPE;
  const bool has_state = state != nullptr;
  if (decode && !has_state) return KDA_ERR_NULL_ARG;
  kda_status_t st = check_seqs(sa, N, rows, P, has_state, decode);
  if (st != KDA_OK) return st;
  if (A_log == nullptr || (rows > 0 && (!x || !dt || !B || !C || !out))) return KDA_ERR_NULL_ARG;
  const int e = elem_size(sh->dtype);
  if (!aligned(x, e) || !aligned(dt, e) || !aligned(B, e) || !aligned(C, e) || !aligned(z, e) ||
      !aligned(out, e) || !aligned(A_log, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) ||
      !aligned(state, 16) || !aligned(steps, 16))
    return KDA_ERR_MISALIGNED;
  const Range rx = rng(x, span(rows, sh->x_stride, Ch, e)),
              rd = rng(dt, span(rows, sh->dt_stride, Ch, e)),
              rz = rng(z, span(rows, sh->z_stride, Ch, e)),
              rB = rng(B, span(rows, sh->b_stride, G * S, e)),
              rC = rng(C, span(rows, sh->c_stride, G * S, e)), rA = rng(A_log, Ch * S * 4),
              rD = rng(D, Ch * 4), rb = rng(dt_bias, Ch * 4), rst = rng(state, P * Ch * S * 4),
              ri = rng(sa.slot, N * 4), rh = rng(sa.has, N),
              rc = rng(sa.cu, (N + 1) * (sa.cu64 ? 8 : 4)), ro = rng(out, rows * Ch * e),
              rp = rng(steps, rows * Ch * S * 4), rs = rng(status, 4);
  for (const Range& o : {ro, rst, rp, rs})
    if (overlap(o, {rx, rd, rz, rB, rC, rA, rD, rb, ri, rh, rc})) return KDA_ERR_OUT_ALIAS;
  if (overlap(ro, {rst, rp, rs}) || overlap(rst, {rp, rs}) || overlap(rp, rs))
    return KDA_ERR_OUT_ALIAS;
  int sms = 0;
  st = device(&sms);
  if (st != KDA_OK) return st;

  ScanParams p{};
  p.x = x;
  p.dt = dt;
  p.B = B;
  p.Cm = C;
  p.z = z;
  p.A_log = A_log;
  p.D = D;
  p.dt_bias = dt_bias;
  p.state = state;
  p.slot = sa.slot;
  p.has = sa.has;
  p.out = out;
  p.steps = steps;
  p.status = status;
  p.seq = make_seqs(sa, N, rows);
  p.xs = sh->x_stride;
  p.ds = sh->dt_stride;
  p.zs = sh->z_stride;
  p.bs = sh->b_stride;
  p.cs = sh->c_stride;
  p.channels = static_cast<int32_t>(Ch);
  p.size = static_cast<int32_t>(S);
  p.groups = static_cast<int32_t>(G);
  p.per_group = static_cast<int32_t>(Ch / G);
  p.pool = static_cast<int32_t>(P);
  p.softplus = (flags & KDA_SCAN_SOFTPLUS) != 0;
  p.keep = (flags & KDA_LAYER_KEEP_STATE) != 0;
  // the longest sequence that there may be: without cu_seqlens known, else at most the hint
  const int64_t max_rows = sa.cu == nullptr ? rows / N
                           : sh->max_seqlen > 0 ? sh->max_seqlen
                                                : rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch(decode ? "kda_scan_decode" : "kda_scan_prefill", [&] {
    return decode ? launch_scan_decode(p, sh->dtype, sms, s)
                  : launch_scan_prefill(p, max_rows, sh->dtype, sms, s);
  });
}

}  // namespace

extern "C" {

kda_status_t kda_conv_prefill(const void* x, const float* weight, const float* bias, void* state,
                              const int32_t* state_indices, const uint8_t* has_state,
                              const void* cu_seqlens, const kda_conv_shape_t* shape, void* out,
                              int32_t* device_status, uint32_t flags, void* stream) {
  const SeqArgs sa{state_indices, has_state, cu_seqlens, device_status,
                   (flags & KDA_LAYER_CU_SEQLENS_I64) != 0};
  return conv_call(x, weight, bias, state, sa, shape, out, nullptr, device_status, flags, false,
                   stream);
}

kda_status_t kda_conv_decode(const void* x, const float* weight, const float* bias, void* state,
                             const int32_t* state_indices, const kda_conv_shape_t* shape,
                             void* out, void* step_states, int32_t* device_status,
                             uint32_t flags, void* stream) {
  const SeqArgs sa{state_indices, nullptr, nullptr, device_status, false};
  return conv_call(x, weight, bias, state, sa, shape, out, step_states, device_status, flags,
                   true, stream);
}

kda_status_t kda_scan_prefill(const void* x, const void* dt, const float* A_log, const void* B,
                              const void* C, const float* D, const void* z,
                              const float* dt_bias, float* state,
                              const int32_t* state_indices, const uint8_t* has_state,
                              const void* cu_seqlens, const kda_scan_shape_t* shape, void* out,
                              int32_t* device_status, uint32_t flags, void* stream) {
  const SeqArgs sa{state_indices, has_state, cu_seqlens, device_status,
                   (flags & KDA_LAYER_CU_SEQLENS_I64) != 0};
  return scan_call(x, dt, A_log, B, C, D, z, dt_bias, state, sa, shape, out, nullptr,
                   device_status, flags, false, stream);
}

kda_status_t kda_scan_decode(const void* x, const void* dt, const float* A_log, const void* B,
                             const void* C, const float* D, const void* z,
                             const float* dt_bias, float* state, const int32_t* state_indices,
                             const kda_scan_shape_t* shape, void* out, float* step_states,
                             int32_t* device_status, uint32_t flags, void* stream) {
  const SeqArgs sa{state_indices, nullptr, nullptr, device_status, false};
  return scan_call(x, dt, A_log, B, C, D, z, dt_bias, state, sa, shape, out, step_states,
                   device_status, flags, true, stream);
}

kda_status_t kda_rms_norm(const void* x, const float* weight, const void* residual,
                          const void* gate, const kda_norm_shape_t* shape, void* out,
                          void* residual_out, float* scales, uint32_t flags, void* stream) {
  if (shape == nullptr) return KDA_ERR_NULL_ARG;
  const kda_norm_shape_t& sh = *shape;
  const bool out8 = sh.out_dtype == KDA_DTYPE_E4M3;
  if ((flags & ~static_cast<uint32_t>(KDA_NORM_GATE_SIGMOID)) || sh.reserved != 0 ||
      !activation_type(sh.dtype) || (!out8 && sh.out_dtype != sh.dtype) ||
      (sh.group != 0 && sh.group != 128) || (!out8 && sh.group != 0) || !(sh.eps >= 0.f) ||
      !std::isfinite(sh.eps))
    return KDA_ERR_BAD_OPTION;
  const int64_t T = sh.tokens, H = sh.heads, W = sh.width, most = int64_t(1) << 40;
  if (T < 0 || H < 1 || W < 1 || W > 32768 || H * W > kMost) return KDA_ERR_BAD_SHAPE;
  if (sh.x_stride < H * W || sh.x_stride > most ||
      (residual && (sh.residual_stride < H * W || sh.residual_stride > most)) ||
      (residual_out && (sh.residual_out_stride < H * W || sh.residual_out_stride > most)) ||
      (gate && (sh.gate_stride < H * W || sh.gate_stride > most)))
    return KDA_ERR_BAD_SHAPE;
  if (T == 0) return KDA_OK;
  if (!x || !out || (out8 && !scales) || (residual_out && !residual)) return KDA_ERR_NULL_ARG;
  if (!out8 && scales) return KDA_ERR_BAD_OPTION;
  const int e = elem_size(sh.dtype);
  if (!aligned(x, e) || !aligned(residual, e) || !aligned(residual_out, e) || !aligned(gate, e) ||
      !aligned(out, out8 ? 1 : e) || !aligned(weight, 4) || !aligned(scales, 4))
    return KDA_ERR_MISALIGNED;
  const int64_t groups = out8 ? (sh.group == 0 ? 1 : (W + 127) / 128) : 0;
  const Range rx = rng(x, span(T, sh.x_stride, H * W, e)), rw = rng(weight, W * 4),
              rr = rng(residual, span(T, sh.residual_stride, H * W, e)),
              rg = rng(gate, span(T, sh.gate_stride, H * W, e)),
              ro = rng(out, T * H * W * (out8 ? 1 : e)),
              rro = rng(residual_out, span(T, sh.residual_out_stride, H * W, e)),
              rs = rng(scales, T * H * groups * 4);
  // in place: a thread has read its elements of a row before it writes them
  const bool out_is_x = out == x && !out8 && sh.x_stride == H * W;
  const bool ro_is_r = residual_out == residual && sh.residual_out_stride == sh.residual_stride;
  const bool ro_is_x = residual_out == x && sh.residual_out_stride == sh.x_stride;
  if (overlap(ro, {rw, rr, rg, rro, rs}) || (overlap(ro, rx) && !out_is_x) ||
      overlap(rro, {rw, rg, rs}) || (overlap(rro, rr) && !ro_is_r) ||
      (overlap(rro, rx) && !ro_is_x) || overlap(rs, {rx, rw, rr, rg}))
    return KDA_ERR_OUT_ALIAS;
  int sms = 0;
  const kda_status_t st = device(&sms);
  if (st != KDA_OK) return st;

  NormParams p{};
  p.x = x;
  p.res = residual;
  p.gate = gate;
  p.weight = weight;
  p.out = out;
  p.res_out = residual_out;
  p.scales = scales;
  p.xs = sh.x_stride;
  p.rs = sh.residual_stride;
  p.ros = sh.residual_out_stride;
  p.gs = sh.gate_stride;
  p.rows = T * H;
  p.heads = sh.heads;
  p.width = sh.width;
  p.group = sh.group;
  p.groups = static_cast<int32_t>(groups);
  p.out8 = out8;
  p.sigmoid = (flags & KDA_NORM_GATE_SIGMOID) != 0;
  const auto rows_of = [&](int n) {      // n elements at a time everywhere
    const int64_t a = n == 8 ? 16 : n * e;
    const auto ok = [&](const void* q, int64_t stride) {
      return q == nullptr || (aligned(q, a) && stride * e % a == 0);
    };
    return W % n == 0 && ok(x, sh.x_stride) && ok(residual, sh.residual_stride) &&
           ok(residual_out, sh.residual_out_stride) && ok(gate, sh.gate_stride) &&
           aligned(out, out8 ? n : a) && aligned(weight, 16);
  };
  p.step = rows_of(8) ? 8 : rows_of(4) ? 4 : 1;
  p.eps = sh.eps;
  p.inv_width = static_cast<float>(1.0 / static_cast<double>(W));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch("kda_rms_norm", [&] { return launch_norm(p, sh.dtype, s); });
}

}  // extern "C"
