// Gradient of the selective scan. With U the gradient of the state after token t and e = -exp(A_log):
//
//   dC_t = S_t^T go_t,  dx_t = dtv U B_t + D go_t,  dB_t = dtv U^T x_t,
//   dl_t = a_t <U, S_{t-1}>,  ddtv = x_t^T U B_t + e dl_t
//
// in blocks of 64 tokens. With l the log-decay summed from the block's start, E_ij = exp(l_i - l_j) for
// j <= i, S the state before the block, U the gradient of the state after it, w_j = exp(l_end - l_j):
//   Gm = C B^T, Pm = go x^T
//   dC_i = sum_j Pm_ij E_ij dtv_j B_j + exp(l_i) S^T go_i
//   dx_j = dtv_j (sum_i Gm_ij E_ij go_i + w_j U B_j) + D go_j
//   dB_j = dtv_j (sum_i Pm_ij E_ij C_i + w_j U^T x_j)
//   dl_t = sum over pairs j < t <= i of F_ij (F = Pm E Gm dtv_j) + sum_{i >= t} exp(l_i) go_i.(S C_i)
//          + sum_{j < t} w_j dtv_j x_j.(U B_j) + exp(l_end) <U, S>

#include "sdm_device.hpp"
#include "sdm_internal.hpp"
#include "sdm_scan.hpp"

namespace sdm {

namespace {

constexpr int Q = 64;  // tokens per block

struct ScanBwdWs {
  float* S;      // [B,H,nb,P,N] states before the blocks
  float* U;      // [B,H,nb,P,N] gradients of the states after them
  double* sums;  // [B,nb,H,3] dA_log, ddt_bias, dD
  int nb;
};

int blocks_of(int T) { return (T + Q - 1) / Q; }

__host__ __device__ inline size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

// One wave per (sequence, head, channel): dir = 0 walks the tokens forward and stores the state
// before every block, dir = 1 backward and stores the gradient of the state after it.
template <bool BF16>
__global__ void __launch_bounds__(256) scan_states_kernel(ScanArgs A, ScanBwdWs W, int dir) {
  const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (u >= (long long)A.B * A.H * A.P) return;
  const int lane = threadIdx.x & 63;
  const int p = (int)(u % A.P), h = (int)(u / A.P % A.H), b = (int)(u / A.P / A.H);
  const int g = h / (A.H / A.G);
  const int n = sequence_length(A.lengths, b, A.T);
  const float rate = -expf(A.A_log[h]), bias = A.dt_bias[h];
  const float* first = dir ? A.ds_out : A.s_in;
  float* out = dir ? W.U : W.S;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (first && lane + 64 * i < A.N) s[i] = first[u * A.N + lane + 64 * i];
  for (int c = 0; c < W.nb; ++c) {
    const int blk = dir ? W.nb - 1 - c : c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane + 64 * i;
      if (k < A.N) out[(((u / A.P) * W.nb + blk) * A.P + p) * A.N + k] = s[i];
    }
    for (int j = 0; j < Q; ++j) {
      const int t = blk * Q + (dir ? Q - 1 - j : j);
      if (t >= n) continue;
      const long long row = (long long)b * A.T + t;
      const float dtv = softplus(A.dt[row * A.ld_dt + h] + bias);
      const float a = expf(fmaxf(rate * dtv, -kMaxDecay));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = lane + 64 * i;
        if (k < A.N) {
          if (dir) {
            const float go = A.go[(((long long)b * A.H + h) * A.T + t) * A.P + p];
            s[i] = a * (s[i] + go * scan_val<BF16>(A.Cm, row * A.ld_c + g * A.N + k));
          } else {
            const float x = scan_val<BF16>(A.x, row * A.ld_x + h * A.P + p);
            s[i] = fmaf(a, s[i], dtv * x * scan_val<BF16>(A.Bm, row * A.ld_b + g * A.N + k));
          }
        }
      }
    }
  }
  if (dir && A.ds_in) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64 * i < A.N) A.ds_in[u * A.N + lane + 64 * i] = s[i];
  }
}

// One workgroup per (sequence, block, group), the group's heads one after the other.
template <bool BF16>
__global__ void __launch_bounds__(256) scan_backward_kernel(ScanArgs A, ScanBwdWs W) {
  __shared__ float Gm[Q][Q + 1], Pm[Q][Q + 1];
  __shared__ double l[Q];
  __shared__ float dtv[Q], slope[Q], read[Q], put[Q], q[Q];
  __shared__ double red[4];
  const int blk = blockIdx.x % W.nb, g = blockIdx.x / W.nb % A.G, b = blockIdx.x / W.nb / A.G;
  const int n = sequence_length(A.lengths, b, A.T);
  const int t0 = blk * Q, tid = threadIdx.x, N = A.N, P = A.P;
  const int here = min(max(n - t0, 0), Q), rows = min(A.T - t0, Q);
  auto xv = [&](int j, int h, int p) { return scan_val<BF16>(A.x, ((long long)b * A.T + t0 + j) * A.ld_x + h * P + p); };
  auto bv = [&](int j, int k) { return scan_val<BF16>(A.Bm, ((long long)b * A.T + t0 + j) * A.ld_b + g * N + k); };
  auto cv = [&](int j, int k) { return scan_val<BF16>(A.Cm, ((long long)b * A.T + t0 + j) * A.ld_c + g * N + k); };
  for (int h = g * (A.H / A.G); h < (g + 1) * (A.H / A.G); ++h) {
    const long long bh = (long long)b * A.H + h;
    const float rate = -expf(A.A_log[h]), D = A.D ? A.D[h] : 0.f;
    const float* S = W.S + (bh * W.nb + blk) * P * N;
    const float* U = W.U + (bh * W.nb + blk) * P * N;
    const float* go = A.go + (bh * A.T + t0) * P;
    __syncthreads();
    if (tid < Q) {
      dtv[tid] = slope[tid] = 0.f;
      if (tid < here) {
        const float raw = A.dt[((long long)b * A.T + t0 + tid) * A.ld_dt + h] + A.dt_bias[h];
        dtv[tid] = softplus(raw);
        slope[tid] = 1.f / (1.f + expf(-raw));
      }
    }
    __syncthreads();
    if (tid == 0) {
      double sum = 0.0;
      for (int j = 0; j < Q; ++j) {
        sum += (double)fmaxf(rate * dtv[j], -kMaxDecay);
        l[j] = sum;
      }
    }
    for (int e = tid; e < here * here; e += 256) {
      const int i = e / here, j = e % here;
      if (j > i) continue;
      float gm = 0.f, pm = 0.f;
      for (int k = 0; k < N; ++k) gm = fmaf(cv(i, k), bv(j, k), gm);
      for (int p = 0; p < P; ++p) pm = fmaf(go[i * P + p], xv(j, h, p), pm);
      Gm[i][j] = gm;
      Pm[i][j] = pm;
    }
    __syncthreads();
    for (int e = tid; e < here * here; e += 256) {
      const int i = e / here, j = e % here;
      if (j > i) continue;
      Pm[i][j] *= (float)exp(l[i] - l[j]);
    }
    __syncthreads();
    // dx
    for (int e = tid; e < rows * P; e += 256) {
      const int j = e / P, p = e % P;
      float s = 0.f;
      if (j < here) {
        float ub = 0.f;
        for (int k = 0; k < N; ++k) ub = fmaf(U[p * N + k], bv(j, k), ub);
        s = (float)exp(l[Q - 1] - l[j]) * ub;
        for (int i = j; i < here; ++i) s = fmaf(Gm[i][j] * (float)exp(l[i] - l[j]), go[i * P + p], s);
        s = fmaf(dtv[j], s, D * go[j * P + p]);
      }
      A.dx[((long long)b * A.T + t0 + j) * A.ld_x + h * P + p] = s;
    }
    // dB and dC, added to those of the heads before
    for (int e = tid; e < rows * N; e += 256) {
      const int j = e / N, k = e % N;
      float db = 0.f, dc = 0.f;
      if (j < here) {
        float ux = 0.f, sg = 0.f;
        for (int p = 0; p < P; ++p) {
          ux = fmaf(U[p * N + k], xv(j, h, p), ux);
          sg = fmaf(S[p * N + k], go[j * P + p], sg);
        }
        db = (float)exp(l[Q - 1] - l[j]) * ux;
        dc = (float)exp(l[j]) * sg;
        for (int i = j; i < here; ++i) db = fmaf(Pm[i][j], cv(i, k), db);
        for (int i = 0; i <= j; ++i) dc = fmaf(Pm[j][i] * dtv[i], bv(i, k), dc);
        db *= dtv[j];
      }
      float* pb = A.dBm + ((long long)b * A.T + t0 + j) * A.ld_b + g * N + k;
      float* pc = A.dCm + ((long long)b * A.T + t0 + j) * A.ld_c + g * N + k;
      const bool add = h > g * (A.H / A.G);
      *pb = add ? *pb + db : db;
      *pc = add ? *pc + dc : dc;
    }
    // gradients of the decay
    float us = 0.f, sd = 0.f;
    for (int e = tid; e < P * N; e += 256) us = fmaf(U[e], S[e], us);
    for (int e = tid; e < here * P; e += 256) sd = fmaf(go[e], xv(e / P, h, e % P), sd);
    us = wave_sum_f32(us);
    sd = wave_sum_f32(sd);
    if ((tid & 63) == 0) red[tid >> 6] = us;
    __syncthreads();
    const double all = red[0] + red[1] + red[2] + red[3];
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = sd;
    if (tid < Q) {
      float r = 0.f, w = 0.f, dq = 0.f;
      if (tid < here) {
        for (int p = 0; p < P; ++p) {
          float sc = 0.f, ub = 0.f;
          for (int k = 0; k < N; ++k) {
            sc = fmaf(S[p * N + k], cv(tid, k), sc);
            ub = fmaf(U[p * N + k], bv(tid, k), ub);
          }
          r = fmaf(go[tid * P + p], sc, r);
          w = fmaf(xv(tid, h, p), ub, w);
        }
        r *= (float)exp(l[tid]);
        w *= (float)exp(l[Q - 1] - l[tid]);
        dq = w;
        for (int i = tid; i < here; ++i) dq = fmaf(Pm[i][tid], Gm[i][tid], dq);
      }
      read[tid] = r;
      put[tid] = w * dtv[tid];
      q[tid] = dq;
    }
    __syncthreads();
    if (tid == 0) {
      double dl = exp(l[Q - 1]) * all, da = 0.0, dbias = 0.0;
      for (int j = 0; j < here; ++j) dl += (double)put[j];
      // from the last token back
      for (int t = here - 1; t >= 0; --t) {
        dl += (double)read[t] - (double)put[t];
        for (int j = 0; j < t; ++j) dl += (double)(Pm[t][j] * Gm[t][j] * dtv[j]);
        for (int i = t + 1; i < here; ++i) dl -= (double)(Pm[i][t] * Gm[i][t] * dtv[t]);
        const double d = ((double)q[t] + dl * rate) * slope[t];
        A.ddt[((long long)b * A.T + t0 + t) * A.ld_dt + h] = (float)d;
        da += dl * rate * dtv[t];
        dbias += d;
      }
      for (int t = here; t < rows; ++t) A.ddt[((long long)b * A.T + t0 + t) * A.ld_dt + h] = 0.f;
      double* out = W.sums + (((long long)b * W.nb + blk) * A.H + h) * 3;
      out[0] = da;
      out[1] = dbias;
      out[2] = red[0] + red[1] + red[2] + red[3];
    }
  }
}

// Sums over sequences and blocks, in their order
__global__ void __launch_bounds__(64) scan_sum_kernel(ScanArgs A, ScanBwdWs W) {
  const int h = blockIdx.x, lane = threadIdx.x;
  double s[3] = {};
  for (long long i = lane; i < (long long)A.B * W.nb; i += 64)
    for (int k = 0; k < 3; ++k) s[k] += W.sums[(i * A.H + h) * 3 + k];
  for (int m = 32; m >= 1; m >>= 1)
    for (int k = 0; k < 3; ++k) s[k] += __shfl_xor(s[k], m, 64);
  if (lane == 0) {
    A.dA_log[h] = (float)s[0];
    A.ddt_bias[h] = (float)s[1];
    if (A.dD) A.dD[h] = (float)s[2];
  }
}

size_t layout(const sdm_scan_shape& S, char* base, ScanBwdWs* W) {
  const size_t nb = blocks_of(S.T), st = round_up((size_t)S.B * S.H * nb * S.d_v * S.d_k * 4);
  W->nb = (int)nb;
  W->S = (float*)base;
  W->U = (float*)(base + st);
  W->sums = (double*)(base + 2 * st);
  return 2 * st + round_up((size_t)S.B * nb * S.H * 3 * 8);
}

}  // namespace

size_t scan_backward_workspace_bytes(const sdm_scan_shape& S) {
  ScanBwdWs W;
  return layout(S, nullptr, &W);
}

hipError_t launch_scan_backward(const sdm_scan_shape& S, const ScanArgs& A, hipStream_t stream) {
  ScanBwdWs W;
  layout(S, (char*)A.ws, &W);
  const dim3 waves((unsigned)(((long long)A.B * A.H * A.P + 3) / 4));
  for (int dir = 0; dir < 2; ++dir) {
    if (A.bf16) hipLaunchKernelGGL(scan_states_kernel<true>, waves, dim3(256), 0, stream, A, W, dir);
    else hipLaunchKernelGGL(scan_states_kernel<false>, waves, dim3(256), 0, stream, A, W, dir);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (W.nb > 0) {
    const dim3 grid((unsigned)((long long)A.B * W.nb * A.G));
    if (A.bf16) hipLaunchKernelGGL(scan_backward_kernel<true>, grid, dim3(256), 0, stream, A, W);
    else hipLaunchKernelGGL(scan_backward_kernel<false>, grid, dim3(256), 0, stream, A, W);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(scan_sum_kernel, dim3(A.H), dim3(64), 0, stream, A, W);
  return hipGetLastError();
}

}  // namespace sdm
