// Passes over the tokens of the selective scan that both its directions share: the time steps and
// decays, and the walk that carries a state (or its gradient) from block to block.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"
#include "sdm_scan.hpp"

namespace sdm {

namespace {

// ------------------------------------------------------------------ time steps
// A workgroup takes 64 tokens of a sequence, all heads: dt comes in along the heads, goes through LDS and
// is summed along the tokens, one per lane. 9 us for 8 x 4096 tokens of 16 heads (one wave per head instead of
// four: 8 us there, but 15 instead of 13 at 131072 tokens of 8).
template <int Q>
__global__ void __launch_bounds__(256) scan_gates_kernel(ScanArgs A, ScanGates g) {
  __shared__ float tile[64][65];
  const int blocks = g.stride / 64, b = blockIdx.x / blocks, t0 = (int)(blockIdx.x % blocks) * 64;
  const int here = min(max(sequence_length(A.lengths, b, A.T) - t0, 0), 64);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int h0 = 0; h0 < A.H; h0 += 64) {
    const int heads = min(A.H - h0, 64);
    __syncthreads();
    for (int i = threadIdx.x; i < here * heads; i += 256)
      tile[i / heads][i % heads] = A.dt[((long long)b * A.T + t0 + i / heads) * A.ld_dt + h0 + i % heads];
    __syncthreads();
    for (int h = wave; h < heads; h += 4) {
      const float step = lane < here ? softplus(tile[lane][h] + A.dt_bias[h0 + h]) : 0.f;
      const float la = lane < here ? fmaxf(-expf(A.A_log[h0 + h]) * step, -kMaxDecay) : 0.f;
      const double l = block_prefix<Q>((double)la * kLog2e);
      const double end = Q == 64 || lane >= 32 ? read_lane(l, 63) : read_lane(l, 31);
      const long long at = ((long long)b * A.H + h0 + h) * g.stride + t0 + lane;
      g.l[at] = l;
      g.step[at] = step;
      g.since[at] = exp2_of(l);
      g.left[at] = exp2_of(end - l) * step;
    }
  }
}

// ------------------------------------------------------------------ the walk
// S' = exp(l_end) S + sum_t (w_t X_t) K_t^T over the blocks of a segment of a (sequence, head, 64 channels)
// unit, the state [d_v, d_k] in the accumulators of its matrix products: wave w holds channels
// 16 w .. 16 w + 15, all d_k. Forward X = x, K = B, w = left; backward, from the last block to the first,
// X = go, K = C, w = since. A block's loads are in flight while the block before is multiplied.
//
// Segments start at zero. With BLOCKS what the segment adds to the state that enters each of its blocks but the
// first is stored (backward: to the gradient of the state after it), and the decay up to there, by which the
// state before the segment, which is known only behind this walk, still has to be multiplied. So one pass over
// the tokens does: a pass for the segments' ends first took 33 us more (4 x 2048 tokens, 8 heads of 128 x 128).
// A walk of one segment starts from the call's state and stores all. Both walks at that size: 42 us, of which
// the 117 MB of states take 24; the forward pass's, without states, is bound like the kernel behind it.
// TURN: results as [channel][d_k] tiles, whose lanes hold 4 consecutive channels, and turned states; else
// the other way round. Each is stored the way the products that read it take it.
constexpr int kPB = 64;

template <int XP, int KP, int NK, bool BACK, bool BLOCKS, bool TURN>
__device__ __forceinline__ void walk(const ScanWalk& A, int id, uint16_t* lds, float* w_) {
  constexpr int Q = KP == 1 ? 64 : 32, NT = 2 * NK;
  constexpr int LX = kPB + 16, LK = NK * 32 + 16, nX = Q * LX, nK = Q * LK;
  uint16_t *Ks = lds, *Xs = Ks + KP * nK;

  const int fast = A.B * A.G * A.segs, hpg = A.H / A.G;
  const int f = id % fast, s = id / fast;
  const int seg = f / (A.B * A.G), b = f % (A.B * A.G) / A.G, g = f % A.G;
  const int h = g * hpg + s % hpg, pb = s / hpg, p0 = pb * kPB;
  const long long bh = (long long)b * A.H + h;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lg = lane >> 4, lr = lane & 15;
  const int n = sequence_length(A.lengths, b, A.T), N = A.N, P = A.P;
  const int s0 = (int)((long long)A.blocks * seg / A.segments), s1 = (int)((long long)A.blocks * (seg + 1) / A.segments);

  // 16-byte pieces: piece i of this thread is in row j + i (256 / pieces-per-row)
  constexpr int XE = XP == 1 ? 8 : 4, KE = KP == 1 ? 8 : 4, XB = XP == 1 ? 2 : 4, KB = KP == 1 ? 2 : 4;
  constexpr int XR = kPB / XE, KR = NK * 32 / KE, NX = Q * XR / 256, NKV = (Q * KR + 255) / 256, XS = 256 / XR, KS = 256 / KR;
  const int xj = tid / XR, xk = (tid % XR) * XE, kj = tid / KR, kk = (tid % KR) * KE;
  const uint32_t xoff = p0 + xk < P ? (uint32_t)(xj * A.ld_x + xk) * XB : kNowhere,
                 koff = kk < N ? (uint32_t)(kj * A.ld_k + kk) * KB : kNowhere;
  const uint32_t xstep = (uint32_t)(XS * A.ld_x) * XB, kstep = (uint32_t)(KS * A.ld_k) * KB;
  const char* px0 = (const char*)A.X + ((long long)b * A.xb + (long long)h * A.xh + p0) * XB;
  const char* pk0 = (const char*)A.K + ((long long)b * A.T * A.ld_k + g * N) * KB;
  const float* pw0 = A.weight + bh * A.stride;
  const double* pl0 = A.l + bh * A.stride;
  // two blocks ahead, in two sets of registers: a block's products are shorter than a load's way
  uint4 rx[2][NX], rk[2][NKV];
  float rw[2] = {0.f, 0.f};
  double rl[2] = {0.0, 0.0};
  auto fetch = [&](int step, int set) {
    // (behind the walk's last block: nothing, but the same loads)
    const int s = min(step, s1 - 1), c = BACK ? A.blocks - 1 - s : s, here = step < s1 ? min(max(n - c * Q, 0), Q) : 0;
    const rsrc_t rows_x = block_rows(px0 + (long long)c * Q * A.ld_x * XB, (uint32_t)(here * A.ld_x) * XB),
                 rows_k = block_rows(pk0 + (long long)c * Q * A.ld_k * KB, (uint32_t)(here * A.ld_k) * KB);
#pragma unroll
    for (int i = 0; i < NX; ++i) rx[set][i] = load16(rows_x, xoff + i * xstep);
#pragma unroll
    for (int i = 0; i < NKV; ++i) rk[set][i] = load16(rows_k, koff + i * kstep);
    rw[set] = pw0[c * Q + (lane & (Q - 1))];
    // (every lane its own: a scalar load's return would be waited for with the next read of LDS)
    rl[set] = pl0[c * Q + (lane & (Q - 1))];
  };
  auto put = [&](uint16_t* tile, int plane, int at, const uint4& v, bool whole) {
    if (whole) {
      *(uint4*)(tile + at) = v;
    } else {
      uint32_t a[3], d[3];
      split_pair(__uint_as_float(v.x), __uint_as_float(v.y), a);
      split_pair(__uint_as_float(v.z), __uint_as_float(v.w), d);
#pragma unroll
      for (int k = 0; k < 3; ++k) *(uint2*)(tile + k * plane + at) = make_uint2(a[k], d[k]);
    }
  };

  // where the four values of tile m lie in a state of the walk's own layout (-1: nowhere)
  auto place = [&](int m) {
    if (TURN) return turned_at(m, P, p0 + 16 * wave + 4 * lg, lr);
    const int p = p0 + 16 * wave + lr, k = 16 * m + 4 * lg;
    return p < P && k < N ? p * N + k : -1;
  };
  const int size = TURN ? turned_size(N, P) : P * N;
  f32x4_t S[NT];
  const float* start = A.segments == 1 && A.start ? A.start + bh * P * N : nullptr;
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    const int at = place(m);
    S[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (TURN && start) {  // [d_v][d_k]
      const int p = p0 + 16 * wave + 4 * lg, k = 16 * m + lr;
      if (p < P && k < N) {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[m][e] = start[(p + e) * N + k];
      }
    } else if (start && at >= 0) {
      S[m] = *(const f32x4_t*)(start + at);
    }
  }
  double total = 0.0;

  auto block = [&](int step, int set) {
    const int c = BACK ? A.blocks - 1 - step : step;
    if (BLOCKS) {
      float* to = A.states + (bh * A.blocks + c) * size;
      // (nothing of a segment's first block, but the same stores)
      const rsrc_t all = block_rows(to, A.segments == 1 || step > s0 ? (uint32_t)size * 4 : 0u);
      if (A.upto && tid == 0 && pb == 0) A.upto[bh * A.blocks + c] = exp2_of(total);
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const int at = place(m);
        store16(all, at >= 0 ? (uint32_t)at * 4 : kNowhere, S[m]);
      }
    }
    __syncthreads();  // the tiles of the block before are read
#pragma unroll
    for (int i = 0; i < NX; ++i) put(Xs, nX, (xj + i * XS) * LX + xk, rx[set][i], XP == 1);
#pragma unroll
    for (int i = 0; i < NKV; ++i)
      if (Q * KR % 256 == 0 || kj + i * KS < Q) put(Ks, nK, (kj + i * KS) * LK + kk, rk[set][i], KP == 1);
    if (wave == 0 && lane < Q) w_[lane] = rw[set];
    const double end = read_lane(rl[set], Q - 1);
    fetch(step + 2, set);
    __syncthreads();
    const float keep = exp2_of(end);
    total += end;
#pragma unroll
    for (int m = 0; m < NT; ++m) S[m] *= keep;
#pragma unroll
    for (int k = 0; k < Q / 32; ++k) {
      float v[8];
      values_of(across<XP>(Xs + 32 * k * LX + 16 * wave, LX, nX, lane), v);
      const f32x4_t w0 = *(const f32x4_t*)(w_ + 32 * k + 4 * lg), w1 = *(const f32x4_t*)(w_ + 32 * k + 16 + 4 * lg);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] *= w0[u];
        v[4 + u] *= w1[u];
      }
      const Frag<3> xw = split8(v);
      constexpr int MH = NT < 4 ? NT : 4;
#pragma unroll
      for (int m = 0; m < NT; m += MH) {
        Frag<KP> kf[MH];
#pragma unroll
        for (int r = 0; r < MH; ++r) kf[r] = across<KP>(Ks + 32 * k * LK + 16 * (m + r), LK, nK, lane);
        if (TURN) mma_rows<MH>(S + m, xw, kf);
        else mma_cols<MH>(S + m, kf, xw);
      }
    }
  };
  if (s0 < s1) fetch(s0, 0);
  if (s0 < s1) fetch(s0 + 1, 1);
  for (int step = s0; step < s1; step += 2) {
    block(step, 0);
    if (step + 1 < s1) block(step + 1, 1);
  }
  float* to = A.segments > 1 ? A.first + ((long long)(seg + 1) * A.B * A.H + bh) * size
              : A.end        ? A.end + bh * P * N
                             : nullptr;
  if (to) {  // (a turned walk of one segment has no end)
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int at = place(m);
      if (at >= 0) *(f32x4_t*)(to + at) = S[m];
    }
  }
  if (A.segments > 1 && tid == 0 && pb == 0) A.decay[(long long)(seg + 1) * A.B * A.H + bh] = total;
}

// The walk for the first states of the forward pass's segments
template <int KP, int NK>
__global__ void __launch_bounds__(256, 2) scan_walk_kernel(ScanWalk A) {
  extern __shared__ __align__(16) uint16_t lds[];
  __shared__ __align__(16) float w_[64];
  walk<KP, KP, NK, false, false, false>(A, blockIdx.x, lds, w_);
}

// The gradient's two walks, which need nothing of each other: workgroups of the longer one, back, come first
template <int KP, int NK>
__global__ void __launch_bounds__(256, 2) scan_walks_kernel(ScanWalk A, ScanWalk U) {
  extern __shared__ __align__(16) uint16_t lds[];
  __shared__ __align__(16) float w_[64];
  const int half = gridDim.x / 2;
  if ((int)blockIdx.x < half) walk<3, KP, NK, true, true, false>(U, blockIdx.x, lds, w_);
  else walk<KP, KP, NK, false, true, true>(A, blockIdx.x - half, lds, w_);
}

// States before the segments, from the segments' own ends: first[0] is the call's first state, first[s]
// (which holds what segment s-1 adds) takes up first[s-1] decayed over segment s-1, and so the call's end.
__device__ __forceinline__ void join(const ScanWalk& A, bool turned, long long group) {
  const long long per = (turned ? turned_size(A.N, A.P) : A.P * A.N) / 4, units = (long long)A.B * A.H;
  const long long i = group * 256 + threadIdx.x;
  if (i >= units * per) return;
  f32x4_t* v = (f32x4_t*)A.first;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (A.start && turned) {
    const int at = (int)(i % per), lane = at % 64, tiles = turned_dv(A.P) / 32;
    const int p = at / 128 % tiles * 32 + lane / 16 * 8 + at / 64 % 2 * 4, k = at / 128 / tiles * 16 + lane % 16;
    if (p < A.P && k < A.N) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = A.start[(i / per * A.P + p + e) * A.N + k];
    }
  } else if (A.start) {
    s = ((const f32x4_t*)A.start)[i];
  }
  v[i] = s;
  const int last = A.segments - (A.end ? 0 : 1);
  for (int k0 = 1; k0 <= last; k0 += 8) {  // eight loads in flight
    f32x4_t add[8];
    float keep[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const long long k = min(k0 + u, last);
      add[u] = v[k * units * per + i];
      keep[u] = exp2_of(A.decay[k * units + i / per]);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k0 + u <= last) {
        s = add[u] + s * keep[u];
        if (k0 + u < A.segments) v[(k0 + u) * units * per + i] = s;
        else ((f32x4_t*)A.end)[i] = s;
      }
  }
}

__global__ void __launch_bounds__(256) scan_join_kernel(ScanWalk A) { join(A, false, blockIdx.x); }
__global__ void __launch_bounds__(256) scan_joins_kernel(ScanWalk A, ScanWalk U, int first) {
  if ((int)blockIdx.x < first) join(A, true, blockIdx.x);
  else join(U, false, blockIdx.x - first);
}

unsigned join_groups(const ScanWalk& A, bool turned) {
  const int size = turned ? turned_size(A.N, A.P) : A.P * A.N;
  return (unsigned)(((long long)A.B * A.H * (size / 4) + 255) / 256);
}
unsigned walk_groups(const ScanWalk& A) { return (unsigned)((long long)A.B * A.H * ((A.P + kPB - 1) / kPB) * A.segs); }
constexpr int walk_lds(int XP, int KP, int NK) {
  return (KP * (KP == 1 ? 64 : 32) * (NK * 32 + 16) + XP * (KP == 1 ? 64 : 32) * (kPB + 16)) * 2;
}

template <int KP, int NK>
hipError_t launch_walk(ScanWalk A, hipStream_t stream) {
  constexpr int lds = walk_lds(KP, KP, NK);
  A.segs = A.segments - 1;
  hipLaunchKernelGGL((scan_walk_kernel<KP, NK>), dim3(walk_groups(A)), dim3(256), lds, stream, A);
  return hipGetLastError();
}

template <int KP, int NK>
hipError_t launch_walks(ScanWalk A, ScanWalk U, hipStream_t stream) {
  constexpr int lds = walk_lds(3, KP, NK);  // (go is float32: three pieces)
  A.segs = U.segs = A.segments;
  hipLaunchKernelGGL((scan_walks_kernel<KP, NK>), dim3(2 * walk_groups(A)), dim3(256), lds, stream, A, U);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_scan_gates(const ScanArgs& A, int Q, const ScanGates& g, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)A.B * (g.stride / 64)));
  if (grid.x == 0) return hipSuccess;
  if (Q == 64) hipLaunchKernelGGL(scan_gates_kernel<64>, grid, dim3(256), 0, stream, A, g);
  else hipLaunchKernelGGL(scan_gates_kernel<32>, grid, dim3(256), 0, stream, A, g);
  return hipGetLastError();
}

hipError_t launch_scan_walk(const ScanWalk& A, bool bf16, hipStream_t stream) {
  hipError_t e = bf16          ? (A.N <= 32   ? launch_walk<1, 1>(A, stream)
                                  : A.N <= 64 ? launch_walk<1, 2>(A, stream)
                                              : launch_walk<1, 4>(A, stream))
                 : A.N <= 32 ? launch_walk<3, 1>(A, stream)
                 : A.N <= 64 ? launch_walk<3, 2>(A, stream)
                             : launch_walk<3, 4>(A, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_join_kernel, dim3(join_groups(A, false)), dim3(256), 0, stream, A);
  return hipGetLastError();
}

hipError_t launch_scan_walks(const ScanWalk& A, const ScanWalk& U, bool bf16, hipStream_t stream) {
  const hipError_t e = bf16          ? (A.N <= 32   ? launch_walks<1, 1>(A, U, stream)
                                        : A.N <= 64 ? launch_walks<1, 2>(A, U, stream)
                                                    : launch_walks<1, 4>(A, U, stream))
                       : A.N <= 32 ? launch_walks<3, 1>(A, U, stream)
                       : A.N <= 64 ? launch_walks<3, 2>(A, U, stream)
                                   : launch_walks<3, 4>(A, U, stream);
  if (e != hipSuccess || A.segments == 1) return e;
  const unsigned first = join_groups(A, true);
  hipLaunchKernelGGL(scan_joins_kernel, dim3(first + join_groups(U, false)), dim3(256), 0, stream, A, U, (int)first);
  return hipGetLastError();
}

}  // namespace sdm
