// Short causal convolution of every channel over the tokens, with its state and its gradient.
//
//   z[t, c] = bias[c] + sum_{j<K} w[c, j] X[t - (K-1) + j, c],   y = z or z sigmoid(z)
// X is x continued into the past by the K-1 inputs of the state. Gradients, with dz = dy act'(z)
// (0 outside the sequence):
//   dX[m] = sum_j w[c, j] dz[m + K-1 - j],  dw[c, j] = sum_t dz[t] X[t - (K-1) + j],  dbias = sum_t dz
// and the last K-1 inputs, which are the state after the call, add ds_out.
//
// About 2 K operations for each value read and written, so memory bounds it. A thread takes 8
// channels (one or two 16-byte accesses a row) of a run of tokens and slides over them with the
// last K rows in registers.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"

namespace sdm {

namespace {

constexpr int kRun = 16;      // tokens per thread
constexpr int kBwdOct = 32;   // backward: channel octets per workgroup
constexpr int kBwdRuns = 8;   // backward: token runs per workgroup

// X[m] of 8 channels for m in [-(K-1), n): the state's rows before token 0, x behind them
template <bool BF16, int K>
__device__ __forceinline__ void load_x(const ConvArgs& A, int b, int m, int c0, float (&v)[8]) {
  if (m >= 0) {
    load8<BF16>(A.x, ((long long)b * A.T + m) * A.ld_x + c0, v);
  } else if (A.s_in && m >= -(K - 1)) {
    load8<BF16>(A.s_in, ((long long)b * (K - 1) + m + K - 1) * A.C + c0, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
}

// ------------------------------------------------------------------ forward
// One thread per (sequence, run, octet), octets fastest. The thread of run 0 also writes the state: it
// alone reads s_in, which may be the same buffer.
template <bool BF16, int K>
__global__ void __launch_bounds__(256) conv_kernel(ConvArgs A, int octets, long long units, int runs) {
  const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int c0 = (int)(u % octets) * 8;
  const int run = (int)(u / octets % runs), b = (int)(u / octets / runs);
  const int n = sequence_length(A.lengths, b, A.T);
  const int t0 = run * kRun;
  float w[K][8], bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bias[e] = A.bias ? A.bias[c0 + e] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][e] = A.w[(long long)(c0 + e) * K + j];
  }
  float win[K][8];  // X[t-(K-1)] .. X[t]
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int m = t0 - (K - 1) + j;
    if (m < n) load_x<BF16, K>(A, b, m, c0, win[j + 1]);
  }
  if (run == 0 && A.s_out) {
    // the last K-1 inputs, all read before the first is written
    float held[K - 1][8];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) load_x<BF16, K>(A, b, n - (K - 1) + i, c0, held[i]);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) store8<BF16>(A.s_out, ((long long)b * (K - 1) + i) * A.C + c0, held[i]);
  }
  const int t1 = min(t0 + kRun, A.T);
  for (int t = t0; t < t1; ++t) {
    float y[8];
    if (t < n) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) win[j][e] = win[j + 1][e];
      load_x<BF16, K>(A, b, t, c0, win[K - 1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) z = fmaf(w[j][e], win[j][e], z);
        y[e] = A.silu ? z / (1.f + expf(-z)) : z;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0.f;
    }
    store8<BF16>(A.y, ((long long)b * A.T + t) * A.ld_y + c0, y);
  }
}

// ------------------------------------------------------------------ backward
// A workgroup takes 32 octets and 8 consecutive runs of one sequence; its sums of dw and dbias
// over those tokens go to one row of `part`, [workgroup][K+1][C].
template <bool BF16, int K>
__global__ void __launch_bounds__(kBwdOct * kBwdRuns) conv_backward_kernel(ConvArgs A, int groups) {
  __shared__ float red[kBwdRuns][kBwdOct * 8];
  const int oct = threadIdx.x % kBwdOct, sub = threadIdx.x / kBwdOct;
  const int c0 = ((int)blockIdx.y * kBwdOct + oct) * 8;
  const int b = (int)(blockIdx.x / groups), group = (int)(blockIdx.x % groups);
  const int t0 = (group * kBwdRuns + sub) * kRun;
  const int n = sequence_length(A.lengths, b, A.T);
  const bool live = c0 < A.C;
  float dw[K][8] = {}, db[8] = {};
  if (live && (t0 < A.T || t0 == 0)) {
    float w[K][8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bias[e] = A.bias ? A.bias[c0 + e] : 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][e] = A.w[(long long)(c0 + e) * K + j];
    }
    float win[K][8], dz[K][8] = {};  // X[t-(K-1)] .. X[t]; dz[t-(K-1)] .. dz[t]
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int m = t0 - (K - 1) + j;
      if (m < n) load_x<BF16, K>(A, b, m, c0, win[j + 1]);
    }
    const int t1 = min(t0 + kRun, A.T);
    for (int t = t0; t < t1 + K - 1; ++t) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          win[j][e] = win[j + 1][e];
          dz[j][e] = dz[j + 1][e];
        }
      if (t < n) {
        load_x<BF16, K>(A, b, t, c0, win[K - 1]);
        float dy[8];
        load8<false>(A.dy, ((long long)b * A.T + t) * A.ld_y + c0, dy);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float g = dy[e];
          if (A.silu) {
            float z = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) z = fmaf(w[j][e], win[j][e], z);
            const float s = 1.f / (1.f + expf(-z));
            g *= s * (1.f + z * (1.f - s));
          }
          dz[K - 1][e] = g;
          if (t < t1) {
            db[e] += g;
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][e] = fmaf(g, win[j][e], dw[j][e]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dz[K - 1][e] = 0.f;
      }
      // dz[m .. m+K-1] are known: dX[m]
      const int m = t - (K - 1);
      if (m < t0 && (t0 > 0 || !A.ds_in)) continue;
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dx[e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dx[e] = fmaf(w[j][e], dz[K - 1 - j][e], dx[e]);
      }
      const int i = m - n + K - 1;  // row of the final state that token m is
      if (A.ds_out && i >= 0 && i < K - 1) {
        float ds[8];
        load8<false>(A.ds_out, ((long long)b * (K - 1) + i) * A.C + c0, ds);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] += ds[e];
      }
      if (m >= 0) store8<false>(A.dx, ((long long)b * A.T + m) * A.ld_x + c0, dx);
      else store8<false>(A.ds_in, ((long long)b * (K - 1) + m + K - 1) * A.C + c0, dx);
    }
  }
  // sums over the workgroup's runs, in their order
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[sub][oct * 8 + e] = j < K ? dw[j < K ? j : 0][e] : db[e];
    __syncthreads();
    const int c = threadIdx.x;  // one channel per thread: kBwdOct * 8 == kBwdOct * kBwdRuns
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kBwdRuns; ++r) s += red[r][c];
    const int ch = (int)blockIdx.y * kBwdOct * 8 + c;
    if (ch < A.C) A.part[((long long)blockIdx.x * (K + 1) + j) * A.C + ch] = s;
  }
}
static_assert(kBwdOct * 8 == kBwdOct * kBwdRuns, "the reduction gives each thread one channel");

// dw[c][j] and dbias[c] from the workgroups' sums, added in their order in float64: 64 columns x 4
// row lanes per workgroup
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* part, float* dw, float* dbias, int C, int K,
                                                       long long n) {
  __shared__ double red[4][64];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane, cols = (K + 1) * C;
  double s = 0.0;
  if (col < cols)
    for (long long i = r; i < n; i += 4) s += (double)part[i * cols + col];
  red[r][lane] = s;
  __syncthreads();
  if (r == 0 && col < cols) {
    const float v = (float)(((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane]);
    const int j = col / C, c = col % C;
    if (j < K) dw[(long long)c * K + j] = v;
    else if (dbias) dbias[c] = v;
  }
}

int conv_bwd_groups(int T) { return T > 0 ? (T + kRun * kBwdRuns - 1) / (kRun * kBwdRuns) : 1; }

template <bool BF16>
hipError_t launch_conv_k(const ConvArgs& A, hipStream_t stream) {
  const int octets = A.C / 8, runs = A.T > 0 ? (A.T + kRun - 1) / kRun : 1;
  const long long units = (long long)octets * runs * A.B;
  const dim3 grid((unsigned)((units + 255) / 256));
  switch (A.K) {
#define SDM_CONV(KK) \
  case KK: hipLaunchKernelGGL((conv_kernel<BF16, KK>), grid, dim3(256), 0, stream, A, octets, units, runs); break;
    SDM_CONV(2) SDM_CONV(3) SDM_CONV(4) SDM_CONV(5) SDM_CONV(6) SDM_CONV(7) SDM_CONV(8)
#undef SDM_CONV
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_conv_backward_k(const ConvArgs& A, hipStream_t stream) {
  const int groups = conv_bwd_groups(A.T);
  const long long blocks = (long long)A.B * groups;
  const dim3 grid((unsigned)blocks, (unsigned)((A.C / 8 + kBwdOct - 1) / kBwdOct));
  switch (A.K) {
#define SDM_CONV(KK)                                                                                              \
  case KK:                                                                                                        \
    hipLaunchKernelGGL((conv_backward_kernel<BF16, KK>), grid, dim3(kBwdOct * kBwdRuns), 0, stream, A, groups); \
    break;
    SDM_CONV(2) SDM_CONV(3) SDM_CONV(4) SDM_CONV(5) SDM_CONV(6) SDM_CONV(7) SDM_CONV(8)
#undef SDM_CONV
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int cols = (A.K + 1) * A.C;
  hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, stream, A.part, A.dw, A.dbias,
                     A.C, A.K, blocks);
  return hipGetLastError();
}

}  // namespace

size_t conv_backward_workspace_bytes(int B, int T, int C, int K) {
  return align_up((size_t)B * conv_bwd_groups(T) * (K + 1) * C * 4);
}

hipError_t launch_conv(const ConvArgs& A, hipStream_t stream) {
  return A.bf16 ? launch_conv_k<true>(A, stream) : launch_conv_k<false>(A, stream);
}

hipError_t launch_conv_backward(const ConvArgs& A, hipStream_t stream) {
  return A.bf16 ? launch_conv_backward_k<true>(A, stream) : launch_conv_backward_k<false>(A, stream);
}

}  // namespace sdm
