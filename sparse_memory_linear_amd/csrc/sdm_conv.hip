// Short causal convolution of every channel over the tokens, with its state and its gradient.
//
//   z[t, c] = bias[c] + sum_{j<K} w[c, j] X[t - (K-1) + j, c],   y = z or z sigmoid(z)
// X is x continued into the past by the K-1 inputs of the state. Gradients, with dz = dy act'(z)
// (0 outside the sequence):
//   dX[m] = sum_j w[c, j] dz[m + K-1 - j],  dw[c, j] = sum_t dz[t] X[t - (K-1) + j],  dbias = sum_t dz
// and the last K-1 inputs, which are the state after the call, add ds_out.
//
// About 2 K operations for each value read and written, so memory bounds it. A thread takes a few channels
// (16-byte accesses) of a run of tokens: four tokens' loads are in flight while the four before are formed
// from the last K-1 + 4 rows, which stay in registers. 8 x 4096 tokens of 1280 bf16 channels: 42 us (168 MB,
// 4.0 TB/s); the gradient of 4 x 2048 tokens of 1536 channels: 33 us.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"

namespace sdm {

namespace {

constexpr int kRun = 16;      // tokens per thread
constexpr int kStep = 4;      // tokens at a time

// W consecutive channels of a row as they lie in memory
template <bool BF16, int W>
struct Row {
  uint32_t q[BF16 ? W / 2 : W];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const char* p = (const char*)base + at * (BF16 ? 2 : 4);
    if (BF16 && W == 4) {
      const uint2 v = *(const uint2*)p;
      q[0] = v.x;
      q[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < (BF16 ? W / 2 : W) / 4; ++i) {
        const uint4 v = *(const uint4*)(p + 16 * i);
        q[4 * i] = v.x;
        q[4 * i + 1] = v.y;
        q[4 * i + 2] = v.z;
        q[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (BF16 ? W / 2 : W); ++i) q[i] = 0u;
  }
  __device__ __forceinline__ float at(int e) const {
    return BF16 ? ((e & 1) ? bf16hi(q[e >> 1]) : bf16lo(q[e >> 1])) : __uint_as_float(q[e]);
  }
};

template <bool BF16>
__device__ __forceinline__ void store4(void* base, long long at, const float (&v)[4]) {
  if (BF16) *(uint2*)((uint16_t*)base + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else *(float4*)((float*)base + at) = make_float4(v[0], v[1], v[2], v[3]);
}

// X[m] of the channels from c0 for m in [-(K-1), n): the state's rows before token 0, x behind them; 0 elsewhere
template <bool BF16, int K, int W>
__device__ __forceinline__ void load_x(const ConvArgs& A, int b, int m, int n, int c0, Row<BF16, W>& r) {
  if (m >= n || (m < 0 && (!A.s_in || m < -(K - 1)))) r.clear();
  else if (m >= 0) r.load(A.x, ((long long)b * A.T + m) * A.ld_x + c0);
  else r.load(A.s_in, ((long long)b * (K - 1) + m + K - 1) * A.C + c0);
}

// ------------------------------------------------------------------ forward
// One thread per (sequence, run, 4 channels), channels fastest: with 8 channels a thread held twice the
// registers and half the waves were resident (48 us against 42 at 8 x 4096 tokens of 1280 channels, for
// 16 bytes a load). The thread of run 0 also writes the state: it
// alone reads s_in, which may be the same buffer.
template <bool BF16, int K>
__global__ void __launch_bounds__(256) conv_kernel(ConvArgs A, int quads, long long units, int runs) {
  const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int c0 = (int)(u % quads) * 4;
  const int run = (int)(u / quads % runs), b = (int)(u / quads / runs);
  const int n = sequence_length(A.lengths, b, A.T);
  const int t0 = run * kRun, t1 = min(t0 + kRun, A.T);
  Row<BF16, 4> next[kStep];
  float win[K - 1 + kStep][4];  // X[t-(K-1)] .. X[t+kStep-1]
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    Row<BF16, 4> r;
    load_x<BF16, K>(A, b, t0 - (K - 1) + j, n, c0, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) win[j][e] = r.at(e);
  }
#pragma unroll
  for (int i = 0; i < kStep; ++i) load_x<BF16, K>(A, b, t0 + i, n, c0, next[i]);
  float w[K][4], bias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = A.bias ? A.bias[c0 + e] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][e] = A.w[(long long)(c0 + e) * K + j];
  }
  if (run == 0 && A.s_out) {
    // the last K-1 inputs, all read before the first is written
    Row<BF16, 4> held[K - 1];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) load_x<BF16, K>(A, b, n - (K - 1) + i, n, c0, held[i]);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = held[i].at(e);
      store4<BF16>(A.s_out, ((long long)b * (K - 1) + i) * A.C + c0, v);
    }
  }
  for (int t = t0; t < t1; t += kStep) {
#pragma unroll
    for (int i = 0; i < kStep; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) win[K - 1 + i][e] = next[i].at(e);
    if (t + kStep < t1) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) load_x<BF16, K>(A, b, t + kStep + i, n, c0, next[i]);
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      if (t + i >= t1) break;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float z = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) z = fmaf(w[j][e], win[i + j][e], z);
        y[e] = t + i < n ? (A.silu ? z * sigmoid_f32(z) : z) : 0.f;
      }
      store4<BF16>(A.y, ((long long)b * A.T + t + i) * A.ld_y + c0, y);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) win[j][e] = win[kStep + j][e];
  }
}

// ------------------------------------------------------------------ backward
// A workgroup takes LANES x 4 channels and RUNS consecutive runs of one sequence; its sums of dw and dbias over
// those tokens go to one row of `part`, [workgroup][K+1][C]. 64 lanes, or 8 for up to 128 channels, which leave
// most of 64 idle (64 x 2048 tokens of 64 channels: 27 us, 53 with 64 lanes).
template <bool BF16, int K, int LANES>
__global__ void __launch_bounds__(256) conv_backward_kernel(ConvArgs A, int groups) {
  constexpr int RUNS = 256 / LANES;
  __shared__ float red[RUNS][LANES * 4];
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const int c0 = ((int)blockIdx.y * LANES + lane) * 4;
  const int b = (int)(blockIdx.x / groups), group = (int)(blockIdx.x % groups);
  const int t0 = (group * RUNS + sub) * kRun;
  const int n = sequence_length(A.lengths, b, A.T);
  const bool live = c0 < A.C;
  float dw[K][4] = {}, db[4] = {};
  if (live && (t0 < A.T || t0 == 0)) {
    const int t1 = min(t0 + kRun, A.T), te = t1 + K - 1;
    Row<BF16, 4> nx[kStep];
    Row<false, 4> ny[kStep];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        load_x<BF16, K>(A, b, t + i, n, c0, nx[i]);
        if (t + i < n) ny[i].load(A.dy, ((long long)b * A.T + t + i) * A.ld_y + c0);
        else ny[i].clear();
      }
    };
    float win[K - 1 + kStep][4], dz[K - 1 + kStep][4];  // X and dz from t-(K-1)
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Row<BF16, 4> r;
      load_x<BF16, K>(A, b, t0 - (K - 1) + j, n, c0, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        win[j][e] = r.at(e);
        dz[j][e] = 0.f;
      }
    }
    fetch(t0);
    float w[K][4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bias[e] = A.bias ? A.bias[c0 + e] : 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][e] = A.w[(long long)(c0 + e) * K + j];
    }
    for (int t = t0; t < te; t += kStep) {
      float dy[kStep][4];
#pragma unroll
      for (int i = 0; i < kStep; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          win[K - 1 + i][e] = nx[i].at(e);
          dy[i][e] = ny[i].at(e);
        }
      if (t + kStep < te) fetch(t + kStep);
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const bool own = t + i < t1;  // (dz of the tokens behind the run only serves dX)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float g = dy[i][e];
          if (A.silu) {
            float z = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) z = fmaf(w[j][e], win[i + j][e], z);
            const float s = sigmoid_f32(z);
            g *= s * (1.f + z * (1.f - s));
          }
          g = t + i < n ? g : 0.f;
          dz[K - 1 + i][e] = g;
          if (own) {
            db[e] += g;
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][e] = fmaf(g, win[i + j][e], dw[j][e]);
          }
        }
        // dz[m .. m+K-1] are known: dX[m]
        const int m = t + i - (K - 1);
        if (m >= t1 || (m < t0 && (t0 > 0 || !A.ds_in))) continue;
        float dx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dx[e] = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) dx[e] = fmaf(w[j][e], dz[K - 1 - j + i][e], dx[e]);
        }
        const int q = m - n + K - 1;  // row of the final state that token m is
        if (A.ds_out && q >= 0 && q < K - 1) {
          const float4 ds = *(const float4*)(A.ds_out + ((long long)b * (K - 1) + q) * A.C + c0);
          dx[0] += ds.x;
          dx[1] += ds.y;
          dx[2] += ds.z;
          dx[3] += ds.w;
        }
        float* to = m >= 0 ? A.dx + ((long long)b * A.T + m) * A.ld_x + c0 : A.ds_in + ((long long)b * (K - 1) + m + K - 1) * A.C + c0;
        *(float4*)to = make_float4(dx[0], dx[1], dx[2], dx[3]);
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          win[j][e] = win[kStep + j][e];
          dz[j][e] = dz[kStep + j][e];
        }
    }
  }
  // sums over the workgroup's runs, in their order; one channel per thread
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[sub][lane * 4 + e] = j < K ? dw[j < K ? j : 0][e] : db[e];
    __syncthreads();
    const int c = threadIdx.x, ch = (int)blockIdx.y * LANES * 4 + c;
    if (c < LANES * 4 && ch < A.C) {
      double s = 0.0;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) s += (double)red[r][c];
      A.part[((long long)blockIdx.x * (K + 1) + j) * A.C + ch] = (float)s;
    }
  }
}

// dw[c][j] and dbias[c] from the workgroups' sums, added in their order in float64: COLS columns x 1024 / COLS
// row lanes per workgroup, eight loads of each in flight. 8 columns where there are many sums of few (540 rows
// and more): of 8192 rows of 24 columns 64 took 50 us more.
template <int COLS>
__global__ void __launch_bounds__(1024) conv_sum_kernel(const float* part, float* dw, float* dbias, int C, int K,
                                                        long long n) {
  constexpr int ROWS = 1024 / COLS;
  __shared__ double red[ROWS][COLS];
  const int lane = threadIdx.x % COLS, r = threadIdx.x / COLS;
  const int col = (int)blockIdx.x * COLS + lane, cols = (K + 1) * C;
  double s = 0.0;
  if (col < cols)
    for (long long i = r; i < n; i += 8 * ROWS) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[min(i + ROWS * u, n - 1) * cols + col];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + ROWS * u < n) s += (double)v[u];
    }
  red[r][lane] = s;
  __syncthreads();
  for (int m = ROWS / 2; m >= 1; m >>= 1) {
    if (r < m) red[r][lane] += red[r + m][lane];
    __syncthreads();
  }
  if (r == 0 && col < cols) {
    const float v = (float)red[0][lane];
    const int j = col / C, c = col % C;
    if (j < K) dw[(long long)c * K + j] = v;
    else if (dbias) dbias[c] = v;
  }
}

int conv_bwd_lanes(int C) { return C <= 128 ? 8 : 64; }
int conv_bwd_groups(int T, int C) {
  const int tokens = kRun * (256 / conv_bwd_lanes(C));
  return T > 0 ? (T + tokens - 1) / tokens : 1;
}

template <bool BF16>
hipError_t launch_conv_k(const ConvArgs& A, hipStream_t stream) {
  const int quads = A.C / 4, runs = A.T > 0 ? (A.T + kRun - 1) / kRun : 1;
  const long long units = (long long)quads * runs * A.B;
  const dim3 grid((unsigned)((units + 255) / 256));
  switch (A.K) {
#define SDM_CONV(KK) \
  case KK: hipLaunchKernelGGL((conv_kernel<BF16, KK>), grid, dim3(256), 0, stream, A, quads, units, runs); break;
    SDM_CONV(2) SDM_CONV(3) SDM_CONV(4) SDM_CONV(5) SDM_CONV(6) SDM_CONV(7) SDM_CONV(8)
#undef SDM_CONV
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_conv_backward_k(const ConvArgs& A, hipStream_t stream) {
  const int groups = conv_bwd_groups(A.T, A.C), lanes = conv_bwd_lanes(A.C);
  const long long blocks = (long long)A.B * groups;
  const dim3 grid((unsigned)blocks, (unsigned)((A.C + lanes * 4 - 1) / (lanes * 4)));
  switch (A.K) {
#define SDM_CONV(KK)                                                                                             \
  case KK:                                                                                                       \
    if (lanes == 8)                                                                                              \
      hipLaunchKernelGGL((conv_backward_kernel<BF16, KK, 8>), grid, dim3(256), 0, stream, A, groups);            \
    else                                                                                                         \
      hipLaunchKernelGGL((conv_backward_kernel<BF16, KK, 64>), grid, dim3(256), 0, stream, A, groups);           \
    break;
    SDM_CONV(2) SDM_CONV(3) SDM_CONV(4) SDM_CONV(5) SDM_CONV(6) SDM_CONV(7) SDM_CONV(8)
#undef SDM_CONV
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int cols = (A.K + 1) * A.C;
  if (blocks > 512 && cols < 64 * 64)
    hipLaunchKernelGGL(conv_sum_kernel<8>, dim3((unsigned)((cols + 7) / 8)), dim3(1024), 0, stream, A.part, A.dw,
                       A.dbias, A.C, A.K, blocks);
  else
    hipLaunchKernelGGL(conv_sum_kernel<64>, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, stream, A.part, A.dw,
                       A.dbias, A.C, A.K, blocks);
  return hipGetLastError();
}

}  // namespace

size_t conv_backward_workspace_bytes(int B, int T, int C, int K) {
  return align_up((size_t)B * conv_bwd_groups(T, C) * (K + 1) * C * 4);
}

hipError_t launch_conv(const ConvArgs& A, hipStream_t stream) {
  return A.bf16 ? launch_conv_k<true>(A, stream) : launch_conv_k<false>(A, stream);
}

hipError_t launch_conv_backward(const ConvArgs& A, hipStream_t stream) {
  return A.bf16 ? launch_conv_backward_k<true>(A, stream) : launch_conv_backward_k<false>(A, stream);
}

}  // namespace sdm
