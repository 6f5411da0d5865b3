// The norms after one layer and before the next, with the gated, scaled residual sum between them,
// and their gradient.
//
//   p = 1 / sqrt(mean(y^2) + eps), yn = y p, u = yn w_post
//   r' = r + scale a u,  a = act(gate)
//   q = 1 / sqrt(mean(r'^2) + eps), h = r' q, x = h w_pre
// Gradients, with t = dx w_pre and s = du w_post:
//   dr' = dr_out + q (t - h mean(t h)),  dr = dr',  du = scale a dr'
//   dgate = scale act'(gate) u dr' over the rows that share it
//   dy = p (s - yn mean(s yn)),  dw_post = sum du yn,  dw_pre = sum dx h
//
// Each value is read once and written once, with a few tens of operations between, so memory
// bounds it: a row stays in the registers of its workgroup between the reductions.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"

namespace sdm {

namespace {

__device__ __forceinline__ void load8_rt(const void* p, bool bf16, long long at, float (&v)[8]) {
  if (bf16) load8<true>(p, at, v);
  else load8<false>(p, at, v);
}
__device__ __forceinline__ void store8_rt(void* p, bool bf16, long long at, const float (&v)[8]) {
  if (bf16) store8<true>(p, at, v);
  else store8<false>(p, at, v);
}

// act(g) and its slope
__device__ __forceinline__ float act_of(int act, float g, float& slope) {
  if (act == SDM_ACT_NONE) {
    slope = 1.f;
    return g;
  }
  const float s = 1.f / (1.f + expf(-g));
  if (act == SDM_ACT_SIGMOID) {
    slope = s * (1.f - s);
    return s;
  }
  slope = s * (1.f + g * (1.f - s));
  return g * s;
}

// 1 / sqrt(v), 0 for 0 (a row of zeros with eps = 0)
__device__ __forceinline__ float inv_rms(float v) { return v > 0.f ? 1.f / sqrtf(v) : (v == 0.f ? 0.f : v); }

// Sum over the workgroup, the same in every thread; `red` holds one value per wave and is free again
// after the caller's next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum_f32(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += red[i];
  return s;
}

// ------------------------------------------------------------------ forward
// A workgroup takes one row at a time; thread i holds octets i, i + blockDim, ... (NC of them).
template <int NC>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs A, long long per_gate) {
  __shared__ float red[2][16];
  const int octets = A.D / 8;
  for (long long m = blockIdx.x; m < A.M; m += gridDim.x) {
    float u[NC][8], r[NC][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        load8_rt(A.y, A.y_bf16, m * A.D + o * 8, u[i]);
        load8_rt(A.r, A.r_bf16, m * A.D + o * 8, r[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(u[i][e], u[i][e], ss);
      }
    }
    float p = 1.f;
    if (A.w_post) p = inv_rms(block_sum(ss, red[0]) / (float)A.D + A.eps);
    float sr = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        if (A.w_post) {
          float w[8];
          load8<false>(A.w_post, o * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] = u[i][e] * p * w[e];
        }
        if (A.gate) {
          float g[8];
          load8_rt(A.gate, A.g_bf16, m / per_gate * A.D + o * 8, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float slope;
            u[i][e] *= act_of(A.act, g[e], slope);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          r[i][e] = fmaf(A.scale, u[i][e], r[i][e]);
          sr = fmaf(r[i][e], r[i][e], sr);
        }
        store8_rt(A.r_out, A.r_bf16, m * A.D + o * 8, r[i]);
      }
    }
    __syncthreads();  // red[0] is free again
    if (!A.x) continue;
    const float q = inv_rms(block_sum(sr, red[1]) / (float)A.D + A.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        float w[8];
        load8<false>(A.w_pre, o * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = r[i][e] * q * w[e];
        store8_rt(A.x, A.x_bf16, m * A.D + o * 8, r[i]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
// Workgroup k of `parts` walks rows [M k / parts, M (k+1) / parts) and keeps their column sums in
// registers. part[k][4][D]: the gate sums of a group of rows that begins before workgroup k's rows
// and ends in them (0) or goes on behind them (1), dw_post (2) and dw_pre (3); a group that lies in
// one workgroup's rows goes straight to dgate.
__device__ __forceinline__ long long part_begin(long long M, int k, int parts) { return M * k / parts; }

template <int NC>
__global__ void __launch_bounds__(1024) norm_backward_kernel(NormArgs A, long long per_gate, int parts) {
  __shared__ float red[4][16];
  const int octets = A.D / 8;
  const int k = blockIdx.x;
  const long long m0 = part_begin(A.M, k, parts), m1 = part_begin(A.M, k + 1, parts);
  float sg[NC][8] = {}, sp[NC][8] = {}, sn[NC][8] = {};
  const float inv = 1.f / (float)A.D;
  for (long long m = m0; m < m1; ++m) {
    float yn[NC][8], h[NC][8], a[NC][8], t[NC][8];
    float ss = 0.f;
    __syncthreads();  // red is free again
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        load8_rt(A.y, A.y_bf16, m * A.D + o * 8, yn[i]);
        load8_rt(A.r, A.r_bf16, m * A.D + o * 8, h[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(yn[i][e], yn[i][e], ss);
      }
    }
    float p = 1.f;
    if (A.w_post) p = inv_rms(block_sum(ss, red[0]) * inv + A.eps);
    float sr = 0.f, st = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        float w[8], g[8], dx[8], wn[8];
        if (A.w_post) load8<false>(A.w_post, o * 8, w);
        if (A.gate) load8_rt(A.gate, A.g_bf16, m / per_gate * A.D + o * 8, g);
        if (A.w_pre) {
          load8<false>(A.dx, m * A.D + o * 8, dx);
          load8<false>(A.w_pre, o * 8, wn);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yn[i][e] *= p;
          float slope = 1.f;
          a[i][e] = A.scale * (A.gate ? act_of(A.act, g[e], slope) : 1.f);
          h[i][e] = fmaf(a[i][e], A.w_post ? yn[i][e] * w[e] : yn[i][e], h[i][e]);  // r'
          t[i][e] = A.w_pre ? dx[e] * wn[e] : 0.f;
          sr = fmaf(h[i][e], h[i][e], sr);
          st = fmaf(t[i][e], h[i][e], st);
        }
      }
    }
    float q = 0.f, mean = 0.f;
    if (A.w_pre) {
      q = inv_rms(block_sum(sr, red[1]) * inv + A.eps);
      mean = block_sum(st, red[2]) * q * inv;  // mean(t h)
    }
    // the last row of its group, or of this workgroup: the gate's sums go out
    const long long grp = m / per_gate, end = (grp + 1) * per_gate;
    const bool flush = A.gate && (m + 1 == end || m + 1 == m1);
    float* gate_to = grp * per_gate >= m0 && end <= m1 ? A.dgate + grp * A.D
                                                       : A.part + ((long long)k * 4 + (end > m1 ? 1 : 0)) * A.D;
    float sy = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
        float w[8], g[8], dx[8], dr[8];
        if (A.dr_out) load8<false>(A.dr_out, m * A.D + o * 8, dr);
        if (A.w_post) load8<false>(A.w_post, o * 8, w);
        if (A.gate) load8_rt(A.gate, A.g_bf16, m / per_gate * A.D + o * 8, g);
        if (A.w_pre) load8<false>(A.dx, m * A.D + o * 8, dx);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[i][e] *= q;
          const float d = (A.dr_out ? dr[e] : 0.f) + q * (t[i][e] - h[i][e] * mean);
          dr[e] = d;
          if (A.w_pre) sn[i][e] = fmaf(dx[e], h[i][e], sn[i][e]);
          const float u = A.w_post ? yn[i][e] * w[e] : yn[i][e];
          float slope = 0.f;
          if (A.gate) act_of(A.act, g[e], slope);
          if (A.gate) sg[i][e] = fmaf(A.scale * slope * u, d, sg[i][e]);
          const float du = a[i][e] * d;
          if (A.w_post) sp[i][e] = fmaf(du, yn[i][e], sp[i][e]);
          t[i][e] = A.w_post ? du * w[e] : du;  // s
          sy = fmaf(t[i][e], yn[i][e], sy);
        }
        store8<false>(A.dr, m * A.D + o * 8, dr);
        if (flush) {
          store8<false>(gate_to, o * 8, sg[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) sg[i][e] = 0.f;
        }
      }
    }
    mean = A.w_post ? block_sum(sy, red[3]) * inv : 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int o = threadIdx.x + i * blockDim.x;
      if (o < octets) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] = A.w_post ? p * (t[i][e] - yn[i][e] * mean) : t[i][e];
        store8<false>(A.dy, m * A.D + o * 8, t[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int o = threadIdx.x + i * blockDim.x;
    if (o < octets) {
      if (A.w_post) store8<false>(A.part, ((long long)k * 4 + 2) * A.D + o * 8, sp[i]);
      if (A.w_pre) store8<false>(A.part, ((long long)k * 4 + 3) * A.D + o * 8, sn[i]);
    }
  }
}

// Column sums of the workgroups, in their order, in float64: dw_post (y = 0), dw_pre (y = 1) and, for
// y = 2 + k, the gate group that begins in workgroup k's rows and goes on behind them, if there is one.
__global__ void __launch_bounds__(256) norm_sum_kernel(NormArgs A, long long per_gate, int parts) {
  __shared__ double red[4][64];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane;
  const int y = (int)blockIdx.y;
  int k0 = 0, k1 = parts;
  long long end = 0;
  float* out = y == 0 ? A.dw_post : A.dw_pre;
  if (y >= 2) {
    k0 = y - 2;
    const long long m0 = part_begin(A.M, k0, parts), m1 = part_begin(A.M, k0 + 1, parts);
    if (m0 == m1) return;
    const long long grp = (m1 - 1) / per_gate;
    end = (grp + 1) * per_gate;
    if (end <= m1 || grp * per_gate < m0) return;  // ends here, or began before
    out = A.dgate + grp * A.D;
    while (k1 > k0 + 1 && part_begin(A.M, k1 - 1, parts) >= end) --k1;
  }
  if (!out) return;
  double s = 0.0;
  if (col < A.D)
    for (int k = k0 + r; k < k1; k += 4) {
      const int slot = y < 2 ? 2 + y : end > part_begin(A.M, k + 1, parts) ? 1 : 0;
      s += (double)A.part[((long long)k * 4 + slot) * A.D + col];
    }
  red[r][lane] = s;
  __syncthreads();
  if (r == 0 && col < A.D) out[col] = (float)(((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane]);
}

// Workgroup width and octets per thread for rows of D values
void row_plan(int D, int* threads, int* nc) {
  const int octets = D / 8;
  *nc = octets > 256 ? 2 : 1;
  int t = (octets + *nc - 1) / *nc;
  t = (t + 63) / 64 * 64;
  *threads = t;
}

// Workgroups of the backward pass: every one has a row
int backward_parts(long long M) { return (int)(M < 1 ? 1 : M < 512 ? M : 512); }

}  // namespace

size_t norm_backward_workspace_bytes(const sdm_norm_shape& S) {
  return align_up((size_t)backward_parts(S.M) * 4 * S.D * 4);
}

hipError_t launch_norm(const NormArgs& A, hipStream_t stream) {
  int threads, nc;
  row_plan(A.D, &threads, &nc);
  const long long per = A.gate_rows > 0 ? A.M / A.gate_rows : 1;
  const dim3 grid((unsigned)(A.M < (1 << 21) ? A.M : (1 << 21))), block((unsigned)threads);
  if (nc == 1) hipLaunchKernelGGL(norm_kernel<1>, grid, block, 0, stream, A, per);
  else hipLaunchKernelGGL(norm_kernel<2>, grid, block, 0, stream, A, per);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& A, hipStream_t stream) {
  int threads, nc;
  row_plan(A.D, &threads, &nc);
  const int parts = backward_parts(A.M);
  const long long per = A.gate_rows > 0 && A.M > 0 ? A.M / A.gate_rows : 1;
  const dim3 grid((unsigned)parts), block((unsigned)threads);
  if (nc == 1) hipLaunchKernelGGL(norm_backward_kernel<1>, grid, block, 0, stream, A, per, parts);
  else hipLaunchKernelGGL(norm_backward_kernel<2>, grid, block, 0, stream, A, per, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (A.M == 0 && A.gate) {
    e = launch_zero(A.dgate, (size_t)A.gate_rows * A.D / 2, stream);
    if (e != hipSuccess) return e;
  }
  const bool gate_sums = A.gate && A.M > 0 && per > 1;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((A.D + 63) / 64), (unsigned)(2 + (gate_sums ? parts : 0))),
                     dim3(256), 0, stream, A, per, parts);
  return hipGetLastError();
}

}  // namespace sdm
