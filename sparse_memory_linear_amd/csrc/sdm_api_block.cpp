// C ABI of the layers around the sparse memory: short convolution, selective scan, block norm.
// As in sdm_api.cpp every check runs on the host before the first HIP call.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/sdm.h"
#include "sdm_internal.hpp"

namespace sdm {

namespace {

constexpr int64_t kMaxTokens = (int64_t)INT32_MAX / 2;
constexpr int64_t kMaxStride = (int64_t)1 << 24;
constexpr int64_t kMaxScanStride = (int64_t)1 << 22;

bool dtype_ok(int dt) { return dt == SDM_F32 || dt == SDM_BF16; }

// One tensor argument: `rows` rows of `width` bytes, `ld` bytes apart.
struct Buf {
  const void* p;
  size_t width, ld;
  int64_t rows;
  bool out;
  bool required;
};

Buf flat(const void* p, size_t bytes, bool out, bool required) { return {p, bytes, bytes, bytes ? 1 : 0, out, required}; }
Buf rows(const void* p, int64_t n, size_t width, int64_t ld, size_t esize, bool out, bool required) {
  return {p, width * esize, (size_t)ld * esize, n, out, required};
}

// Do two tensors share a byte? Slices of the columns of one wide buffer (the same distance
// between rows) are apart if their columns are.
bool share(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.rows == 0 || b.rows == 0) return false;
  const size_t na = (size_t)(a.rows - 1) * a.ld + a.width, nb = (size_t)(b.rows - 1) * b.ld + b.width;
  if (!overlaps(a.p, na, b.p, nb)) return false;
  if (a.ld != b.ld || a.rows < 2 || b.rows < 2) return true;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  const size_t d = pb >= pa ? (pb - pa) % a.ld : (a.ld - (pa - pb) % a.ld) % a.ld;
  return d < a.width || d + b.width > a.ld;
}

// Null, alignment and overlap checks: outputs apart from every other tensor, except the pair
// (same0, same1), which may be one and the same buffer.
sdm_status check_bufs(const Buf* b, int n, int same0 = -1, int same1 = -1) {
  for (int i = 0; i < n; ++i) {
    if (!b[i].p && b[i].required && b[i].rows > 0) return SDM_ERR_INVALID_ARG;
    if (!aligned16(b[i].p)) return SDM_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!b[i].out && !b[j].out) continue;
      if (i == same0 && j == same1 && b[i].p == b[j].p) continue;
      if (share(b[i], b[j])) return SDM_ERR_INVALID_ARG;
    }
  return SDM_OK;
}

// ------------------------------------------------------------------ shapes
sdm_status check_conv(const sdm_conv_shape* S) {
  if (!S) return SDM_ERR_INVALID_ARG;
  if (S->B < 1 || S->T < 0 || S->C < 1 || S->K < 1) return SDM_ERR_INVALID_ARG;
  if (!dtype_ok(S->in_dtype)) return SDM_ERR_INVALID_ARG;
  if (S->act != SDM_ACT_NONE && S->act != SDM_ACT_SILU) return SDM_ERR_INVALID_ARG;
  if (S->ld_x < S->C || S->ld_y < S->C) return SDM_ERR_INVALID_ARG;
  if (S->K < 2 || S->K > 8 || S->C % 8 != 0 || S->ld_x % 8 != 0 || S->ld_y % 8 != 0) return SDM_ERR_UNSUPPORTED;
  if (S->C > (1 << 20) || S->ld_x > kMaxStride || S->ld_y > kMaxStride) return SDM_ERR_UNSUPPORTED;
  if ((int64_t)S->B * S->T > kMaxTokens) return SDM_ERR_UNSUPPORTED;
  // grids: one thread per 16 tokens of 4 channels, one workgroup per 64 tokens
  if ((int64_t)S->B * (S->T / 16 + 1) > ((int64_t)1 << 31) / (S->C / 4) ||
      (int64_t)S->B * (S->T / 64 + 1) > (1 << 23))
    return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

sdm_status check_scan(const sdm_scan_shape* S) {
  if (!S) return SDM_ERR_INVALID_ARG;
  if (S->B < 1 || S->T < 0 || S->H < 1 || S->G < 1 || S->H % S->G != 0) return SDM_ERR_INVALID_ARG;
  if (S->d_k < 1 || S->d_v < 1 || !dtype_ok(S->in_dtype)) return SDM_ERR_INVALID_ARG;
  if (S->H > 4096 || S->d_k > 128 || S->d_v > 256 || S->d_k % 8 != 0 || S->d_v % 8 != 0) return SDM_ERR_UNSUPPORTED;
  if (S->ld_x < (int64_t)S->H * S->d_v || S->ld_b < (int64_t)S->G * S->d_k || S->ld_c < (int64_t)S->G * S->d_k ||
      S->ld_dt < S->H)
    return SDM_ERR_INVALID_ARG;
  if (S->ld_x % 8 != 0 || S->ld_b % 8 != 0 || S->ld_c % 8 != 0) return SDM_ERR_UNSUPPORTED;
  // a block of 64 rows is addressed with 32-bit byte offsets
  if (S->ld_x > kMaxScanStride || S->ld_b > kMaxScanStride || S->ld_c > kMaxScanStride || S->ld_dt > kMaxScanStride)
    return SDM_ERR_UNSUPPORTED;
  if ((int64_t)S->B * S->T > (kMaxTokens >> 1) || (int64_t)S->B * S->H > 65535) return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

// The gradient's grids: one workgroup per block of 32 tokens and head at most
sdm_status check_scan_backward(const sdm_scan_shape* S) {
  const sdm_status st = check_scan(S);
  if (st != SDM_OK) return st;
  return (int64_t)S->B * (S->T / 32 + 1) * S->H > (1 << 22) ? SDM_ERR_UNSUPPORTED : SDM_OK;
}

sdm_status check_norm(const sdm_norm_shape* S) {
  if (!S) return SDM_ERR_INVALID_ARG;
  if (S->M < 0 || S->D < 1 || S->gate_rows < 0) return SDM_ERR_INVALID_ARG;
  if (!dtype_ok(S->y_dtype) || !dtype_ok(S->r_dtype) || !dtype_ok(S->x_dtype) || !dtype_ok(S->gate_dtype))
    return SDM_ERR_INVALID_ARG;
  if (S->gate_act != SDM_ACT_NONE && S->gate_act != SDM_ACT_SILU && S->gate_act != SDM_ACT_SIGMOID)
    return SDM_ERR_INVALID_ARG;
  if (S->gate_rows > 0 && S->M % S->gate_rows != 0) return SDM_ERR_INVALID_ARG;
  if (!(S->eps >= 0.f) || S->eps > 1.f || !isfinite(S->scale)) return SDM_ERR_INVALID_ARG;
  if (S->D % 8 != 0 || S->D > 16384 || S->M > kMaxTokens) return SDM_ERR_UNSUPPORTED;
  // gate_rows divides M, so it is at most M unless M is 0
  if (S->gate_rows > kMaxTokens) return SDM_ERR_UNSUPPORTED;
  return SDM_OK;
}

sdm_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return SDM_OK;
  if (!ws || ws_bytes < need) return SDM_ERR_WORKSPACE;
  return aligned16(ws) ? SDM_OK : SDM_ERR_INVALID_ARG;
}

ConvArgs conv_args(const sdm_conv_shape& S) {
  ConvArgs A{};
  A.B = S.B;
  A.T = S.T;
  A.C = S.C;
  A.K = S.K;
  A.ld_x = S.ld_x;
  A.ld_y = S.ld_y;
  A.bf16 = S.in_dtype == SDM_BF16;
  A.silu = S.act == SDM_ACT_SILU;
  return A;
}

sdm_status conv_impl(const sdm_conv_shape* S, const void* x, const float* w, const float* bias, const int32_t* lengths,
                     const void* s_in, void* s_out, void* y, void* stream) {
  const size_t e = dtype_size(S->in_dtype);
  const int64_t n = (int64_t)S->B * S->T;
  const size_t held = (size_t)S->B * (S->K - 1) * S->C * e;
  const Buf b[] = {flat(s_in, held, false, false),
                   flat(s_out, held, true, false),
                   rows(x, n, S->C, S->ld_x, e, false, true),
                   flat(w, (size_t)S->C * S->K * 4, false, true),
                   flat(bias, (size_t)S->C * 4, false, false),
                   flat(lengths, (size_t)S->B * 4, false, false),
                   rows(y, n, S->C, S->ld_y, e, true, true)};
  const sdm_status st = check_bufs(b, 7, 0, 1);
  if (st != SDM_OK) return st;
  if (n == 0 && !s_out) return SDM_OK;
  ConvArgs A = conv_args(*S);
  A.x = x;
  A.w = w;
  A.bias = bias;
  A.lengths = lengths;
  A.s_in = s_in;
  A.s_out = s_out;
  A.y = y;
  return hip_status(launch_conv(A, (hipStream_t)stream));
}

ScanArgs scan_args(const sdm_scan_shape& S, const void* x, const void* Bm, const void* Cm, const float* dt,
                   const float* A_log, const float* dt_bias, const float* D) {
  ScanArgs A{};
  A.B = S.B;
  A.T = S.T;
  A.H = S.H;
  A.G = S.G;
  A.N = S.d_k;
  A.P = S.d_v;
  A.ld_x = S.ld_x;
  A.ld_b = S.ld_b;
  A.ld_c = S.ld_c;
  A.ld_dt = S.ld_dt;
  A.bf16 = S.in_dtype == SDM_BF16;
  A.x = x;
  A.Bm = Bm;
  A.Cm = Cm;
  A.dt = dt;
  A.A_log = A_log;
  A.dt_bias = dt_bias;
  A.D = D;
  return A;
}

size_t scan_state_bytes(const sdm_scan_shape& S) { return (size_t)S.B * S.H * S.d_v * S.d_k * 4; }
size_t scan_out_bytes(const sdm_scan_shape& S) { return (size_t)S.B * S.H * (size_t)S.T * S.d_v * 4; }

}  // namespace

}  // namespace sdm

using namespace sdm;

extern "C" {

// ------------------------------------------------------------------ short convolution
sdm_status sdm_check_conv_shape(const sdm_conv_shape* shape) { return check_conv(shape); }

sdm_status sdm_short_conv(const sdm_conv_shape* S, const void* x, const float* w, const float* bias,
                          const int32_t* lengths, const void* s_in, void* s_out, void* y, void* stream) {
  const sdm_status st = check_conv(S);
  if (st != SDM_OK) return st;
  return conv_impl(S, x, w, bias, lengths, s_in, s_out, y, stream);
}

sdm_status sdm_short_conv_step(const sdm_conv_shape* S, const void* x, const float* w, const float* bias, void* state,
                               void* y, void* stream) {
  const sdm_status st = check_conv(S);
  if (st != SDM_OK) return st;
  if (S->T != 1 || !state) return SDM_ERR_INVALID_ARG;
  return conv_impl(S, x, w, bias, nullptr, state, state, y, stream);
}

size_t sdm_short_conv_backward_workspace_bytes(const sdm_conv_shape* S) {
  if (check_conv(S) != SDM_OK) return 0;
  return conv_backward_workspace_bytes(S->B, S->T, S->C, S->K);
}

sdm_status sdm_short_conv_backward(const sdm_conv_shape* S, const void* x, const float* w, const float* bias,
                                   const int32_t* lengths, const void* s_in, const float* dy, const float* ds_out,
                                   float* dx, float* dw, float* dbias, float* ds_in, void* ws, size_t ws_bytes,
                                   void* stream) {
  sdm_status st = check_conv(S);
  if (st != SDM_OK) return st;
  if ((bias != nullptr) != (dbias != nullptr)) return SDM_ERR_INVALID_ARG;
  const size_t need = conv_backward_workspace_bytes(S->B, S->T, S->C, S->K);
  st = check_ws(ws, ws_bytes, need);
  if (st != SDM_OK) return st;
  const size_t e = dtype_size(S->in_dtype);
  const int64_t n = (int64_t)S->B * S->T;
  const size_t held = (size_t)S->B * (S->K - 1) * S->C;
  const Buf b[] = {rows(x, n, S->C, S->ld_x, e, false, true),
                   flat(w, (size_t)S->C * S->K * 4, false, true),
                   flat(bias, (size_t)S->C * 4, false, false),
                   flat(lengths, (size_t)S->B * 4, false, false),
                   flat(s_in, held * e, false, false),
                   rows(dy, n, S->C, S->ld_y, 4, false, true),
                   flat(ds_out, held * 4, false, false),
                   rows(dx, n, S->C, S->ld_x, 4, true, true),
                   flat(dw, (size_t)S->C * S->K * 4, true, true),
                   flat(dbias, (size_t)S->C * 4, true, false),
                   flat(ds_in, held * 4, true, false),
                   flat(ws, ws ? need : 0, true, false)};
  st = check_bufs(b, 12);
  if (st != SDM_OK) return st;
  ConvArgs A = conv_args(*S);
  A.x = x;
  A.w = w;
  A.bias = bias;
  A.lengths = lengths;
  A.s_in = s_in;
  A.dy = dy;
  A.ds_out = ds_out;
  A.dx = dx;
  A.dw = dw;
  A.dbias = dbias;
  A.ds_in = ds_in;
  A.part = (float*)ws;
  return hip_status(launch_conv_backward(A, (hipStream_t)stream));
}

// ------------------------------------------------------------------ selective scan
sdm_status sdm_check_scan_shape(const sdm_scan_shape* shape) { return check_scan(shape); }

size_t sdm_selective_scan_workspace_bytes(const sdm_scan_shape* S) {
  return check_scan(S) == SDM_OK ? scan_workspace_bytes(*S) : 0;
}

sdm_status sdm_selective_scan(const sdm_scan_shape* S, const void* x, const void* Bm, const void* Cm, const float* dt,
                              const float* A_log, const float* dt_bias, const float* D, const int32_t* lengths,
                              const float* s_in, float* s_out, float* o, void* ws, size_t ws_bytes, void* stream) {
  sdm_status st = check_scan(S);
  if (st != SDM_OK) return st;
  const size_t need = scan_workspace_bytes(*S);
  st = check_ws(ws, ws_bytes, need);
  if (st != SDM_OK) return st;
  const size_t e = dtype_size(S->in_dtype);
  const int64_t n = (int64_t)S->B * S->T;
  const Buf b[] = {flat(s_in, scan_state_bytes(*S), false, false),
                   flat(s_out, scan_state_bytes(*S), true, false),
                   rows(x, n, (size_t)S->H * S->d_v, S->ld_x, e, false, true),
                   rows(Bm, n, (size_t)S->G * S->d_k, S->ld_b, e, false, true),
                   rows(Cm, n, (size_t)S->G * S->d_k, S->ld_c, e, false, true),
                   rows(dt, n, S->H, S->ld_dt, 4, false, true),
                   flat(A_log, (size_t)S->H * 4, false, true),
                   flat(dt_bias, (size_t)S->H * 4, false, true),
                   flat(D, (size_t)S->H * 4, false, false),
                   flat(lengths, (size_t)S->B * 4, false, false),
                   flat(o, scan_out_bytes(*S), true, true),
                   flat(need ? ws : nullptr, need, true, false)};
  st = check_bufs(b, 12, 0, 1);
  if (st != SDM_OK) return st;
  if (n == 0 && !s_out) return SDM_OK;
  ScanArgs A = scan_args(*S, x, Bm, Cm, dt, A_log, dt_bias, D);
  A.lengths = lengths;
  A.s_in = s_in;
  A.s_out = s_out;
  A.o = o;
  A.ws = ws;
  return hip_status(launch_scan(*S, A, (hipStream_t)stream));
}

sdm_status sdm_selective_scan_step(const sdm_scan_shape* S, const void* x, const void* Bm, const void* Cm,
                                   const float* dt, const float* A_log, const float* dt_bias, const float* D,
                                   float* state, float* o, void* stream) {
  sdm_status st = check_scan(S);
  if (st != SDM_OK) return st;
  if (S->T != 1) return SDM_ERR_INVALID_ARG;
  const size_t e = dtype_size(S->in_dtype);
  const Buf b[] = {flat(state, scan_state_bytes(*S), true, true),
                   rows(x, S->B, (size_t)S->H * S->d_v, S->ld_x, e, false, true),
                   rows(Bm, S->B, (size_t)S->G * S->d_k, S->ld_b, e, false, true),
                   rows(Cm, S->B, (size_t)S->G * S->d_k, S->ld_c, e, false, true),
                   rows(dt, S->B, S->H, S->ld_dt, 4, false, true),
                   flat(A_log, (size_t)S->H * 4, false, true),
                   flat(dt_bias, (size_t)S->H * 4, false, true),
                   flat(D, (size_t)S->H * 4, false, false),
                   flat(o, scan_out_bytes(*S), true, true)};
  st = check_bufs(b, 9);
  if (st != SDM_OK) return st;
  ScanArgs A = scan_args(*S, x, Bm, Cm, dt, A_log, dt_bias, D);
  A.s_in = state;
  A.s_out = state;
  A.o = o;
  return hip_status(launch_scan_step(A, (hipStream_t)stream));
}

size_t sdm_selective_scan_backward_workspace_bytes(const sdm_scan_shape* S) {
  return check_scan_backward(S) == SDM_OK ? scan_backward_workspace_bytes(*S) : 0;
}

sdm_status sdm_selective_scan_backward(const sdm_scan_shape* S, const void* x, const void* Bm, const void* Cm,
                                       const float* dt, const float* A_log, const float* dt_bias, const float* D,
                                       const int32_t* lengths, const float* s_in, const float* go, const float* ds_out,
                                       float* dx, float* dBm, float* dCm, float* ddt, float* dA_log, float* ddt_bias,
                                       float* dD, float* ds_in, void* ws, size_t ws_bytes, void* stream) {
  sdm_status st = check_scan_backward(S);
  if (st != SDM_OK) return st;
  if ((D != nullptr) != (dD != nullptr)) return SDM_ERR_INVALID_ARG;
  const size_t need = scan_backward_workspace_bytes(*S);
  st = check_ws(ws, ws_bytes, need);
  if (st != SDM_OK) return st;
  const size_t e = dtype_size(S->in_dtype), hb = (size_t)S->H * 4;
  const int64_t n = (int64_t)S->B * S->T;
  const size_t xw = (size_t)S->H * S->d_v, kw = (size_t)S->G * S->d_k;
  const Buf b[] = {rows(x, n, xw, S->ld_x, e, false, true),
                   rows(Bm, n, kw, S->ld_b, e, false, true),
                   rows(Cm, n, kw, S->ld_c, e, false, true),
                   rows(dt, n, S->H, S->ld_dt, 4, false, true),
                   flat(A_log, hb, false, true),
                   flat(dt_bias, hb, false, true),
                   flat(D, hb, false, false),
                   flat(lengths, (size_t)S->B * 4, false, false),
                   flat(s_in, scan_state_bytes(*S), false, false),
                   flat(go, scan_out_bytes(*S), false, true),
                   flat(ds_out, scan_state_bytes(*S), false, false),
                   rows(dx, n, xw, S->ld_x, 4, true, true),
                   rows(dBm, n, kw, S->ld_b, 4, true, true),
                   rows(dCm, n, kw, S->ld_c, 4, true, true),
                   rows(ddt, n, S->H, S->ld_dt, 4, true, true),
                   flat(dA_log, hb, true, true),
                   flat(ddt_bias, hb, true, true),
                   flat(dD, hb, true, false),
                   flat(ds_in, scan_state_bytes(*S), true, false),
                   flat(ws, ws ? need : 0, true, false)};
  st = check_bufs(b, 20);
  if (st != SDM_OK) return st;
  ScanArgs A = scan_args(*S, x, Bm, Cm, dt, A_log, dt_bias, D);
  A.lengths = lengths;
  A.s_in = s_in;
  A.go = go;
  A.ds_out = ds_out;
  A.dx = dx;
  A.dBm = dBm;
  A.dCm = dCm;
  A.ddt = ddt;
  A.dA_log = dA_log;
  A.ddt_bias = ddt_bias;
  A.dD = dD;
  A.ds_in = ds_in;
  A.ws = ws;
  return hip_status(launch_scan_backward(*S, A, (hipStream_t)stream));
}

// ------------------------------------------------------------------ block norm
sdm_status sdm_check_norm_shape(const sdm_norm_shape* shape) { return check_norm(shape); }

namespace {
NormArgs norm_args(const sdm_norm_shape& S) {
  NormArgs A{};
  A.M = S.M;
  A.gate_rows = S.gate_rows;
  A.D = S.D;
  A.y_bf16 = S.y_dtype == SDM_BF16;
  A.r_bf16 = S.r_dtype == SDM_BF16;
  A.x_bf16 = S.x_dtype == SDM_BF16;
  A.g_bf16 = S.gate_dtype == SDM_BF16;
  A.act = S.gate_act;
  A.eps = S.eps;
  A.scale = S.scale;
  return A;
}
}  // namespace

sdm_status sdm_block_norm(const sdm_norm_shape* S, const void* y, const void* r, const void* gate, const float* w_post,
                          const float* w_pre, void* r_out, void* x, void* stream) {
  sdm_status st = check_norm(S);
  if (st != SDM_OK) return st;
  if ((S->M > 0 && (x != nullptr) != (w_pre != nullptr)) || (gate != nullptr) != (S->gate_rows > 0))
    return SDM_ERR_INVALID_ARG;
  const size_t n = (size_t)S->M * S->D, wb = (size_t)S->D * 4;
  const Buf b[] = {flat(r, n * dtype_size(S->r_dtype), false, true),
                   flat(r_out, n * dtype_size(S->r_dtype), true, true),
                   flat(y, n * dtype_size(S->y_dtype), false, true),
                   flat(gate, (size_t)S->gate_rows * S->D * dtype_size(S->gate_dtype), false, false),
                   flat(w_post, wb, false, false),
                   flat(w_pre, wb, false, false),
                   flat(x, n * dtype_size(S->x_dtype), true, false)};
  st = check_bufs(b, 7, 0, 1);
  if (st != SDM_OK) return st;
  if (S->M == 0) return SDM_OK;
  NormArgs A = norm_args(*S);
  A.y = y;
  A.r = r;
  A.gate = gate;
  A.w_post = w_post;
  A.w_pre = w_pre;
  A.r_out = r_out;
  A.x = x;
  return hip_status(launch_norm(A, (hipStream_t)stream));
}

size_t sdm_block_norm_backward_workspace_bytes(const sdm_norm_shape* S) {
  return check_norm(S) == SDM_OK ? norm_backward_workspace_bytes(*S) : 0;
}

sdm_status sdm_block_norm_backward(const sdm_norm_shape* S, const void* y, const void* r, const void* gate,
                                   const float* w_post, const float* w_pre, const float* dr_out, const float* dx,
                                   float* dy, float* dr, float* dgate, float* dw_post, float* dw_pre, void* ws,
                                   size_t ws_bytes, void* stream) {
  sdm_status st = check_norm(S);
  if (st != SDM_OK) return st;
  if ((gate != nullptr) != (S->gate_rows > 0) || (dgate != nullptr) != (gate != nullptr) ||
      (dw_post != nullptr) != (w_post != nullptr) || (dw_pre != nullptr) != (w_pre != nullptr) ||
      (S->M > 0 && (dx != nullptr) != (w_pre != nullptr)))
    return SDM_ERR_INVALID_ARG;
  const size_t need = norm_backward_workspace_bytes(*S);
  st = check_ws(ws, ws_bytes, need);
  if (st != SDM_OK) return st;
  const size_t n = (size_t)S->M * S->D, wb = (size_t)S->D * 4, gn = (size_t)S->gate_rows * S->D;
  const Buf b[] = {flat(dr_out, n * 4, false, false),
                   flat(dr, n * 4, true, true),
                   flat(y, n * dtype_size(S->y_dtype), false, true),
                   flat(r, n * dtype_size(S->r_dtype), false, true),
                   flat(gate, gn * dtype_size(S->gate_dtype), false, false),
                   flat(w_post, wb, false, false),
                   flat(w_pre, wb, false, false),
                   flat(dx, n * 4, false, false),
                   flat(dy, n * 4, true, true),
                   flat(dgate, gn * 4, true, false),
                   flat(dw_post, wb, true, false),
                   flat(dw_pre, wb, true, false),
                   flat(ws, ws ? need : 0, true, false)};
  st = check_bufs(b, 13, 0, 1);
  if (st != SDM_OK) return st;
  NormArgs A = norm_args(*S);
  A.y = y;
  A.r = r;
  A.gate = gate;
  A.w_post = w_post;
  A.w_pre = w_pre;
  A.dr_out = dr_out;
  A.dx = dx;
  A.dy = dy;
  A.dr = dr;
  A.dgate = dgate;
  A.dw_post = dw_post;
  A.dw_pre = dw_pre;
  A.part = (float*)ws;
  return hip_status(launch_norm_backward(A, (hipStream_t)stream));
}

}  // extern "C"
