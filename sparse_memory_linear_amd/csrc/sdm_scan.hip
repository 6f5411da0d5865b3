// Selective state space scan: a dense state per head that decays by a scalar of the token and takes
// up an outer product of the token's channels and its B, read through its C.
//
//   dtv = softplus(dt + dt_bias), a = exp(-exp(A_log) dtv)
//   S_t = a_t S_{t-1} + dtv_t x_t B_t^T,   o_t = S_t C_t + D x_t

#include "sdm_device.hpp"
#include "sdm_internal.hpp"
#include "sdm_scan.hpp"

namespace sdm {

namespace {

// One wave per (sequence, head, channel): its row of the state in registers, token after token.
template <bool BF16>
__global__ void __launch_bounds__(256) scan_seq_kernel(ScanArgs A) {
  const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= (long long)A.B * A.H * A.P) return;
  const int lane = threadIdx.x & 63;
  const int p = (int)(u % A.P), h = (int)(u / A.P % A.H), b = (int)(u / A.P / A.H);
  const int g = h / (A.H / A.G);
  const int n = sequence_length(A.lengths, b, A.T);
  const float rate = -expf(A.A_log[h]), bias = A.dt_bias[h], D = A.D ? A.D[h] : 0.f;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (A.s_in && lane + 64 * i < A.N) s[i] = A.s_in[u * A.N + lane + 64 * i];
  for (int t = 0; t < A.T; ++t) {
    float o = 0.f;
    if (t < n) {
      const long long row = (long long)b * A.T + t;
      const float dtv = softplus(A.dt[row * A.ld_dt + h] + bias);
      const float a = expf(fmaxf(rate * dtv, -kMaxDecay));
      const float x = scan_val<BF16>(A.x, row * A.ld_x + h * A.P + p);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = lane + 64 * i;
        if (k < A.N) {
          s[i] = fmaf(a, s[i], dtv * x * scan_val<BF16>(A.Bm, row * A.ld_b + g * A.N + k));
          o = fmaf(s[i], scan_val<BF16>(A.Cm, row * A.ld_c + g * A.N + k), o);
        }
      }
      o = wave_sum_f32(o) + D * x;
    }
    if (lane == 0) A.o[(((long long)b * A.H + h) * A.T + t) * A.P + p] = o;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (A.s_out && lane + 64 * i < A.N) A.s_out[u * A.N + lane + 64 * i] = s[i];
}

}  // namespace

size_t scan_workspace_bytes(const sdm_scan_shape&) { return 0; }

hipError_t launch_scan(const sdm_scan_shape&, const ScanArgs& A, hipStream_t stream) {
  const long long units = (long long)A.B * A.H * A.P;
  const dim3 grid((unsigned)((units + 3) / 4));
  if (A.bf16) hipLaunchKernelGGL(scan_seq_kernel<true>, grid, dim3(256), 0, stream, A);
  else hipLaunchKernelGGL(scan_seq_kernel<false>, grid, dim3(256), 0, stream, A);
  return hipGetLastError();
}

hipError_t launch_scan_step(const ScanArgs& A, hipStream_t stream) { return launch_scan(sdm_scan_shape{}, A, stream); }

}  // namespace sdm
