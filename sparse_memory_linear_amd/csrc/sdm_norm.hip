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
// bounds it: a row stays in the registers of its workgroup between the reductions. Forward, 32768 rows of 2048
// (805 MB): 142 us, 5.7 TB/s. Gradient, 8192 rows of 1536 (277 MB): 75 us, 66 of them the rows and 9 the sums
// over workgroups; without the next row's loads under way 87.

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
  const float s = sigmoid_f32(g);
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

// The same for rows of up to 256 values: L lanes hold a row, a wave 64 / L of them (65536 x 16 rows of 64, 805 MB:
// 144 us; 560 with a wave per row).
template <int L>
__global__ void __launch_bounds__(256) norm_narrow_kernel(NormArgs A, long long per_gate) {
  constexpr int ROWS = 256 / L;
  const int lane = threadIdx.x % L, o = lane * 8;
  const bool in = o < A.D;
  auto row_sum = [](float v) {
#pragma unroll
    for (int k = L / 2; k >= 1; k >>= 1) v = add_xor_f32(v, k);
    return v;
  };
  float w_post[8] = {}, w_pre[8] = {};
  if (in && A.w_post) load8<false>(A.w_post, o, w_post);
  if (in && A.w_pre) load8<false>(A.w_pre, o, w_pre);
  for (long long m0 = (long long)blockIdx.x * ROWS; m0 < A.M; m0 += (long long)gridDim.x * ROWS) {
    const long long m = m0 + threadIdx.x / L;
    const bool live = in && m < A.M;
    float u[8] = {}, r[8] = {}, g[8] = {};
    if (live) {
      load8_rt(A.y, A.y_bf16, m * A.D + o, u);
      load8_rt(A.r, A.r_bf16, m * A.D + o, r);
      if (A.gate) load8_rt(A.gate, A.g_bf16, m / per_gate * A.D + o, g);
    }
    if (A.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
      const float p = inv_rms(row_sum(ss) / (float)A.D + A.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = u[e] * p * w_post[e];
    }
    float sr = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float slope;
      if (A.gate) u[e] *= act_of(A.act, g[e], slope);
      r[e] = fmaf(A.scale, u[e], r[e]);
      sr = fmaf(r[e], r[e], sr);
    }
    if (live) store8_rt(A.r_out, A.r_bf16, m * A.D + o, r);
    if (!A.x) continue;
    const float q = inv_rms(row_sum(sr) / (float)A.D + A.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = r[e] * q * w_pre[e];
    if (live) store8_rt(A.x, A.x_bf16, m * A.D + o, r);
  }
}

// ------------------------------------------------------------------ backward
// Workgroup k of `parts` takes rows [M k / parts, M (k+1) / parts) and keeps their column sums in
// registers. WPR waves hold a row between them, or L lanes of one (196608 rows of 64: 62 us with 8, 263 with 64),
// NC octets a lane; a workgroup's row slots take its rows in turn, so that with a wave or less a row no wave waits
// for another. part[k][4][D]: the gate sums of a group of
// rows that begins before workgroup k's rows and ends in them (0) or goes on behind them (1), dw_post (2)
// and dw_pre (3); a group that lies in one workgroup's rows goes straight to dgate.
__device__ __forceinline__ long long part_begin(long long M, int k, int parts) { return M * k / parts; }

template <int NC, int WPR, int L = 64>
__global__ void __launch_bounds__(WPR > 4 ? 64 * WPR : 256, WPR > 8 ? 4 : NC * WPR > 4 ? 2 : 3) norm_backward_kernel(NormArgs A, long long per_gate, int parts) {
  constexpr int WAVES = WPR > 4 ? WPR : 4, LANES = WPR > 1 ? 64 * WPR : L, SLOTS = 64 * WAVES / LANES;
  __shared__ float red[2][3][WAVES][2];  // by the row's parity: a row may have one meeting only
  int turn = 0;
  __shared__ __align__(16) float sums[SLOTS > 1 ? SLOTS * LANES * NC * 8 : 1];
  const int octets = A.D / 8, wave = threadIdx.x >> 6, slot = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int k = blockIdx.x;
  const long long m0 = part_begin(A.M, k, parts), m1 = part_begin(A.M, k + 1, parts);
  const float inv = 1.f / (float)A.D;
  // sums of two values over a row, the same in all its lanes
  auto row_sum = [&](float& v, float& w, int which) {
#pragma unroll
    for (int k = (LANES < 64 ? LANES : 64) / 2; k >= 1; k >>= 1) {
      v = add_xor_f32(v, k);
      w = add_xor_f32(w, k);
    }
    if (WPR > 1) {
      if ((threadIdx.x & 63) == 0) {
        red[turn][which][wave][0] = v;
        red[turn][which][wave][1] = w;
      }
      __syncthreads();
      v = w = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        v += red[turn][which][slot * WPR + i][0];
        w += red[turn][which][slot * WPR + i][1];
      }
    }
  };
  // column sums over the slots, in their order, to `to`
  auto flush = [&](const float (&s)[NC][8], float* to) {
    if (SLOTS > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[((slot * NC + i) * LANES + lane) * 8 + e] = s[i][e];
      __syncthreads();
      for (int q = threadIdx.x; q < octets * 2; q += 64 * WAVES) {  // 4 columns each
        const int o = q >> 1, at = (o / LANES * LANES + o % LANES) * 8 + (q & 1) * 4;
        float4 v = *(const float4*)(sums + at);
        for (int r = 1; r < SLOTS; ++r) {
          const float4 w = *(const float4*)(sums + r * NC * LANES * 8 + at);
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        *(float4*)(to + o * 8 + (q & 1) * 4) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (lane + i * LANES < octets) store8<false>(to, (lane + i * LANES) * 8, s[i]);
    }
  };

  // A row's values as they lie in memory: with one octet a lane the next row's are under way while a row is
  // worked on, and the weights stay
  constexpr bool AHEAD = NC == 1;
  struct Octet {
    uint4 a, b;  // (bf16: a)
  } ry[NC], rr[NC], rt[NC], rd[NC];
  auto fetch = [&](long long mm, long long row) {  // row mm + .. of the rows from mm (the same for all; -1: none)
    const int below = (int)(row - mm);
    auto row_of = [&](const void* base, bool bf16, bool there) {
      return block_rows((const char*)base + mm * A.D * (bf16 ? 2 : 4), there && mm >= 0 ? (uint32_t)(SLOTS * A.D) * (bf16 ? 2 : 4) : 0u);
    };
    auto octet = [&](rsrc_t r, bool bf16, int o) {
      const uint32_t at = o < octets ? (uint32_t)(below * octets + o) * (bf16 ? 16 : 32) : kNowhere;
      return Octet{load16(r, at), load16(r, bf16 ? kNowhere : at + 16)};
    };
    const rsrc_t y = row_of(A.y, A.y_bf16, true), r = row_of(A.r, A.r_bf16, true), x = row_of(A.dx, false, A.w_pre != nullptr),
                 d = row_of(A.dr_out, false, A.dr_out != nullptr);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      ry[i] = octet(y, A.y_bf16, lane + i * LANES);
      rr[i] = octet(r, A.r_bf16, lane + i * LANES);
      rt[i] = octet(x, false, lane + i * LANES);
      rd[i] = octet(d, false, lane + i * LANES);
    }
  };
  auto values = [](const Octet& q, bool bf16, float (&v)[8]) {
    const float f[8] = {__uint_as_float(q.a.x), __uint_as_float(q.a.y), __uint_as_float(q.a.z), __uint_as_float(q.a.w),
                        __uint_as_float(q.b.x), __uint_as_float(q.b.y), __uint_as_float(q.b.z), __uint_as_float(q.b.w)};
    const float h[8] = {bf16lo(q.a.x), bf16hi(q.a.x), bf16lo(q.a.y), bf16hi(q.a.y),
                        bf16lo(q.a.z), bf16hi(q.a.z), bf16lo(q.a.w), bf16hi(q.a.w)};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bf16 ? h[e] : f[e];
  };
  float kept_post[8] = {}, kept_pre[8] = {};
  if (AHEAD && lane < octets) {
    if (A.w_post) load8<false>(A.w_post, lane * 8, kept_post);
    if (A.w_pre) load8<false>(A.w_pre, lane * 8, kept_pre);
  }
  auto weight = [&](const float* all, const float (&kept)[8], int o, float (&v)[8]) {
    if (!AHEAD) {
      if (all) load8<false>(all, o * 8, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = kept[e];
    }
  };

  float sg[NC][8] = {}, sp[NC][8] = {}, sn[NC][8] = {};
  const bool summed = A.gate && per_gate > 1;  // a gate of each token has no sums
  auto group_end = [&](long long g0) {
    const long long end = summed ? (g0 / per_gate + 1) * per_gate : m1;
    return end < m1 ? end : m1;
  };
  auto row_at = [&](long long mm, long long g1) { return mm + slot < g1 ? mm + slot : g1 - 1; };
  if (AHEAD && m0 < m1) fetch(m0, row_at(m0, group_end(m0)));
  for (long long g0 = m0; g0 < m1;) {
    const long long grp = g0 / per_gate, end = summed ? (grp + 1) * per_gate : m1, g1 = group_end(g0);
    for (long long mm = g0; mm < g1; mm += SLOTS) {
      const bool live = mm + slot < g1;
      const long long m = row_at(mm, g1);  // (behind the last: that again, for nothing)
      const long long gate_row = (summed ? grp : m) * A.D;  // (without sums: a gate of each token)
      turn ^= 1;
      float yn[NC][8], h[NC][8], t[NC][8], dr[NC][8];
      float ss = 0.f, none = 0.f;
      if (!AHEAD) fetch(mm, m);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int o = lane + i * LANES;
        if (o < octets) {
          values(ry[i], A.y_bf16, yn[i]);
          values(rr[i], A.r_bf16, h[i]);
          values(rt[i], false, t[i]);
          values(rd[i], false, dr[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(yn[i][e], yn[i][e], ss);
        }
      }
      if (AHEAD) {
        const long long next = mm + SLOTS < g1 ? mm + SLOTS : g1 < m1 ? g1 : -1;
        fetch(next, next < 0 ? next : row_at(next, next < g1 ? g1 : group_end(next)));
      }
      float p = 1.f;
      if (A.w_post) {
        row_sum(ss, none, 0);
        p = inv_rms(ss * inv + A.eps);
      }
      float sr = 0.f, st = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int o = lane + i * LANES;
        if (o < octets) {
          float w[8], g[8], wn[8];
          weight(A.w_post, kept_post, o, w);
          weight(A.w_pre, kept_pre, o, wn);
          if (A.gate) load8_rt(A.gate, A.g_bf16, gate_row + o * 8, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            yn[i][e] *= p;
            float slope = 1.f;
            const float a = A.scale * (A.gate ? act_of(A.act, g[e], slope) : 1.f);
            h[i][e] = fmaf(a, A.w_post ? yn[i][e] * w[e] : yn[i][e], h[i][e]);  // r'
            if (A.w_pre) st = fmaf(t[i][e] * wn[e], h[i][e], st);
            sr = fmaf(h[i][e], h[i][e], sr);
          }
        }
      }
      float q = 0.f, mean = 0.f;
      if (A.w_pre) {
        row_sum(sr, st, 1);
        q = inv_rms(sr * inv + A.eps);
        mean = st * q * inv;  // mean(t h)
      }
      float sy = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int o = lane + i * LANES;
        if (o < octets) {
          float w[8], g[8], wn[8], dg[8];
          weight(A.w_post, kept_post, o, w);
          weight(A.w_pre, kept_pre, o, wn);
          if (A.gate) load8_rt(A.gate, A.g_bf16, gate_row + o * 8, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float d = dr[i][e];
            if (A.w_pre) {
              const float hn = h[i][e] * q;
              d += q * (t[i][e] * wn[e] - hn * mean);
              if (live) sn[i][e] = fmaf(t[i][e], hn, sn[i][e]);
            }
            dr[i][e] = d;
            const float u = A.w_post ? yn[i][e] * w[e] : yn[i][e];
            float slope = 0.f, a = A.scale;
            if (A.gate) a *= act_of(A.act, g[e], slope);
            dg[e] = A.scale * slope * u * d;
            if (summed && live) sg[i][e] += dg[e];
            const float du = a * d;
            if (A.w_post && live) sp[i][e] = fmaf(du, yn[i][e], sp[i][e]);
            t[i][e] = A.w_post ? du * w[e] : du;  // s
            sy = fmaf(t[i][e], yn[i][e], sy);
          }
          if (live) {
            store8<false>(A.dr, m * A.D + o * 8, dr[i]);
            if (A.gate && !summed) store8<false>(A.dgate, m * A.D + o * 8, dg);
          }
        }
      }
      if (A.w_post) row_sum(sy, none, 2);
      mean = sy * inv;
      if (live) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int o = lane + i * LANES;
          if (o < octets) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[i][e] = A.w_post ? p * (t[i][e] - yn[i][e] * mean) : t[i][e];
            store8<false>(A.dy, m * A.D + o * 8, t[i]);
          }
        }
      }
    }
    if (summed) {
      flush(sg, grp * per_gate >= m0 && end <= m1 ? A.dgate + grp * A.D : A.part + ((long long)k * 4 + (end > m1 ? 1 : 0)) * A.D);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[i][e] = 0.f;
    }
    g0 = g1;
  }
  if (A.w_post) flush(sp, A.part + ((long long)k * 4 + 2) * A.D);
  if (A.w_pre) flush(sn, A.part + ((long long)k * 4 + 3) * A.D);
}

// Column sums of the workgroups, in their order, in float64: dw_post (y = 0), dw_pre (y = 1) and, for
// y >= 2, a gate group that workgroups share: group y - 2 (BY_GROUP: fewer groups than workgroups), or the one
// that begins in the rows of workgroup y - 2 and goes on behind them, if there is one.
// 64 columns x 16 row lanes, eight loads of each in flight: 512 rows are four round trips.
template <bool BY_GROUP>
__global__ void __launch_bounds__(1024) norm_sum_kernel(NormArgs A, long long per_gate, int parts) {
  __shared__ double red[16][64];
  const int lane = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 64 + lane;
  const int y = (int)blockIdx.y;
  int k0 = 0, k1 = parts;
  long long end = 0;
  float* out = y == 0 ? A.dw_post : A.dw_pre;
  if (y >= 2) {
    long long grp = y - 2;
    if (BY_GROUP) {
      // the workgroup that holds its first row
      k0 = (int)(grp * per_gate * parts / A.M);
      while (k0 + 1 < parts && part_begin(A.M, k0 + 1, parts) <= grp * per_gate) ++k0;
      end = (grp + 1) * per_gate;
      if (end <= part_begin(A.M, k0 + 1, parts)) return;  // no other holds any
    } else {
      k0 = y - 2;
      const long long m0 = part_begin(A.M, k0, parts), m1 = part_begin(A.M, k0 + 1, parts);
      if (m0 == m1) return;
      grp = (m1 - 1) / per_gate;
      end = (grp + 1) * per_gate;
      if (end <= m1 || grp * per_gate < m0) return;  // ends here, or began before
    }
    out = A.dgate + grp * A.D;
    // the workgroup that holds its last row
    k1 = (int)min((long long)parts, (end - 1) * parts / A.M + 2);
    while (k1 > k0 + 1 && part_begin(A.M, k1 - 1, parts) >= end) --k1;
  }
  if (!out) return;
  double s = 0.0;
  if (col < A.D)
    for (int kk = k0 + r; kk < k1; kk += 128) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = min(kk + 16 * u, k1 - 1);
        const int slot = y < 2 ? 2 + y : end > part_begin(A.M, k + 1, parts) ? 1 : 0;
        v[u] = A.part[((long long)k * 4 + slot) * A.D + col];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (kk + 16 * u < k1) s += (double)v[u];
    }
  red[r][lane] = s;
  __syncthreads();
  if (r == 0 && col < A.D) {
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    out[col] = (float)s;
  }
}

// Workgroup width and octets per thread for rows of D values
void row_plan(int D, int* threads, int* nc) {
  const int octets = D / 8;
  *nc = octets > 256 ? 2 : 1;
  int t = (octets + *nc - 1) / *nc;
  t = (t + 63) / 64 * 64;
  *threads = t;
}

// Workgroups of the backward pass: as many as are resident at once (three per compute unit while four waves
// hold a row or several, one of 8 or 16), so that few partial sums are written (1536 rows of 8192: 101 us, 113
// with two of 8 waves per compute unit, of which one waits); every one has a row
int backward_parts(long long M, int D) {
  const int most = D <= 2048 ? 768 : 256;
  return (int)(M < 1 ? 1 : M < most ? M : most);
}

}  // namespace

size_t norm_backward_workspace_bytes(const sdm_norm_shape& S) {
  return align_up((size_t)backward_parts(S.M, S.D) * 4 * S.D * 4);
}

hipError_t launch_norm(const NormArgs& A, hipStream_t stream) {
  const long long per = A.gate_rows > 0 ? A.M / A.gate_rows : 1;
  if (A.D <= 256) {
    const int lanes = A.D <= 64 ? 8 : A.D <= 128 ? 16 : 32;
    const long long groups = (A.M * lanes + 255) / 256;
    const dim3 grid((unsigned)(groups < (1 << 21) ? groups : (1 << 21)));
    if (lanes == 8) hipLaunchKernelGGL(norm_narrow_kernel<8>, grid, dim3(256), 0, stream, A, per);
    else if (lanes == 16) hipLaunchKernelGGL(norm_narrow_kernel<16>, grid, dim3(256), 0, stream, A, per);
    else hipLaunchKernelGGL(norm_narrow_kernel<32>, grid, dim3(256), 0, stream, A, per);
    return hipGetLastError();
  }
  int threads, nc;
  row_plan(A.D, &threads, &nc);
  const dim3 grid((unsigned)(A.M < (1 << 21) ? A.M : (1 << 21))), block((unsigned)threads);
  if (nc == 1) hipLaunchKernelGGL(norm_kernel<1>, grid, block, 0, stream, A, per);
  else hipLaunchKernelGGL(norm_kernel<2>, grid, block, 0, stream, A, per);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& A, hipStream_t stream) {
  const int parts = backward_parts(A.M, A.D), octets = A.D / 8;
  const long long per = A.gate_rows > 0 && A.M > 0 ? A.M / A.gate_rows : 1;
#define SDM_NORM(NC, WPR)                                                                                            \
  hipLaunchKernelGGL((norm_backward_kernel<NC, WPR>), dim3((unsigned)parts), dim3(WPR > 4 ? 64 * WPR : 256), 0, stream, \
                     A, per, parts)
#define SDM_NORM_NARROW(L)                                                                                           \
  hipLaunchKernelGGL((norm_backward_kernel<1, 1, L>), dim3((unsigned)parts), dim3(256), 0, stream, A, per, parts)
  if (octets <= 8) SDM_NORM_NARROW(8);
  else if (octets <= 16) SDM_NORM_NARROW(16);
  else if (octets <= 32) SDM_NORM_NARROW(32);
  else if (octets <= 64) SDM_NORM(1, 1);
  else if (octets <= 128) SDM_NORM(1, 2);
  else if (octets <= 256) SDM_NORM(1, 4);
  else if (octets <= 512) SDM_NORM(1, 8);
  else if (octets <= 1024) SDM_NORM(2, 8);
  else SDM_NORM(2, 16);
#undef SDM_NORM
#undef SDM_NORM_NARROW
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (A.M == 0 && A.gate) {
    e = launch_zero(A.dgate, (size_t)A.gate_rows * A.D / 2, stream);
    if (e != hipSuccess) return e;
  }
  const int cols = (A.D + 63) / 64;
  const bool gate_sums = A.gate && A.M > 0 && per > 1;
  if (gate_sums && A.gate_rows >= parts)
    hipLaunchKernelGGL(norm_sum_kernel<false>, dim3(cols, 2 + parts), dim3(1024), 0, stream, A, per, parts);
  else
    hipLaunchKernelGGL(norm_sum_kernel<true>, dim3(cols, 2 + (gate_sums ? (int)A.gate_rows : 0)), dim3(1024), 0, stream, A, per,
                       parts);
  return hipGetLastError();
}

}  // namespace sdm
