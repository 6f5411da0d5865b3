// Gradient of the selective scan. With U the gradient of the state after token t and e = -exp(A_log):
//
//   dC_t = S_t^T go_t,  dx_t = step U B_t + D go_t,  dB_t = step U^T x_t,
//   dl_t = a_t <U, S_{t-1}>,  dstep_t = x_t^T U B_t + e dl_t
//
// in blocks of Q tokens. With l the log-decay summed from the block's start, E_ij = exp(l_i - l_j) for
// j <= i, S the state before the block, U the gradient of the state after it, w_j = exp(l_end - l_j):
//   G = C B^T, P = go x^T,  M_ij = G_ij E_ij step_j,  R_ij = P_ij E_ij step_j
//   dx_j = sum_i M_ij go_i + w_j step_j U B_j + D go_j
//   dC_i = sum_j R_ij B_j + exp(l_i) S^T go_i,   dB_j = sum_i R_ij C_i + w_j step_j U^T x_j
//   dl_t = sum over pairs j < t <= i of F_ij step_j + sum_{i >= t} read_i + sum_{j < t} step_j put_j
//          + exp(l_end) <U, S>
//   with F_ij = P_ij E_ij G_ij, read_i = exp(l_i) C_i . S^T go_i, put_j = w_j B_j . U^T x_j
//   x_j^T U_j B_j = sum_{i >= j} F_ij + put_j
// The pairs' sum over a token is a difference of sums over rows and columns of F: both are taken in
// float64 of the same float32 F, so that what is on both sides cancels.
//
// Three steps: the states S of all blocks (a walk over x and B), the gradients U (a walk over go and C from
// the end), then every block by itself. A workgroup of 8 waves takes one block of one group and some of its
// heads, one after the other, and sums their dB and dC in registers; G is formed once. Every product runs on
// the matrix cores with float32 factors as three bf16 pieces.
//
// 4 x 2048 tokens, 8 heads of 128 x 128: 151 us, of which the blocks take 93, the walks 42, their join 8, the
// sums 6, gates 5. The blocks' matrix work takes 20% of their time and their vector work 45%: LDS (142 KB) holds
// one workgroup per compute unit, whose 8 waves meet about ten times a head.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"
#include "sdm_scan.hpp"

namespace sdm {

namespace {

constexpr int kPB = 64;       // channels per tile
constexpr int kWaves = 8, kThreads = 64 * kWaves;

struct ScanBwd {
  // The states before the blocks and the gradients behind them, in segments of blocks: what the segment adds,
  // [B*H][blocks] of turned states and of [P][N], and, of several segments, the states before those,
  // [segments][B*H], and the factors they take for the block, [B*H][blocks]
  const float *S, *U, *S_first, *U_first, *S_upto, *U_upto;
  int segments;
  double* sums;    // [B*blocks][H][3]: dA_log, ddt_bias, dD of the block
  float* part;     // [parts][2][B*T][G*N]: dC and dB of the parts' heads (parts > 1)
  int blocks, parts, heads;  // heads per part
};

template <bool BF16, int NK>
struct BwdTiles {
  static constexpr int Q = BF16 ? 64 : 32, NP = BF16 ? 1 : 3, QT = Q / 16, NT = 2 * NK;
  static constexpr int LB = NK * 32 + 16, LX = kPB + 16, LM = Q + 8, LU = NK * 32 + 16;
  static constexpr int nB = Q * LB, nX = Q * LX, nM = Q * LM, nU = kPB * LU;
  static constexpr int shared = nU > 2 * nM ? 3 * nU : 6 * nM;  // U takes the place of M and R
  static constexpr int bytes = (2 * NP * nB + (NP + 3) * nX + shared) * 2;
  static constexpr int MT = QT * (QT + 1) / 2;  // tiles of M on and below the diagonal
};

template <bool BF16, int NK>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_kernel(ScanArgs A, ScanGates R, ScanBwd W) {
  using TL = BwdTiles<BF16, NK>;
  constexpr int Q = TL::Q, NP = TL::NP, QT = TL::QT, NT = TL::NT, MT = TL::MT;
  constexpr int LB = TL::LB, LX = TL::LX, LM = TL::LM, LU = TL::LU, nB = TL::nB, nX = TL::nX, nM = TL::nM, nU = TL::nU;
  extern __shared__ __align__(16) uint16_t lds[];
  __shared__ __align__(16) double l_[Q], row_[2][MT][16], col_[2][MT][16], us_[kWaves];
  __shared__ __align__(16) float step_[Q], since_[Q], left_[Q], w_[Q], up_[Q], diag_[2][Q], trace_[2][Q];
  __shared__ __align__(16) float read_[NT][Q], put_[NT][Q];
  uint16_t *Bs = lds, *Cs = Bs + NP * nB, *Xs = Cs + NP * nB, *Gs = Xs + NP * nX, *Ms = Gs + 3 * nX, *Rs = Ms + 3 * nM,
           *Us = Ms;

  int id = blockIdx.x;
  const int part = id % W.parts;
  id /= W.parts;
  const int g = id % A.G;
  id /= A.G;
  const int blk = id % W.blocks, b = id / W.blocks;
  const int hpg = A.H / A.G, h0 = g * hpg + part * W.heads, h1 = min(h0 + W.heads, (g + 1) * hpg);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int tid = threadIdx.x, lane = tid & 63, lg = lane >> 4, lr = lane & 15;
  // Where a stage begins: its addresses are made from the thread's index anew. Kept over the loops they would
  // not fit the registers, and a reload of one waits for every load and store under way.
  auto anew = [&] {
    asm volatile("" : "+v"(tid));
    lane = tid & 63;
    lg = lane >> 4;
    lr = lane & 15;
  };
  const int N = A.N, P = A.P, t0 = blk * Q, n = sequence_length(A.lengths, b, A.T);
  const int here = min(max(n - t0, 0), Q), rows = min(A.T - t0, Q);
  const long long row0 = (long long)b * A.T + t0;
  const int pblocks = (P + kPB - 1) / kPB;

  // where the sums of dC and dB go
  const long long ldc = W.parts > 1 ? (long long)A.G * N : A.ld_c, ldb = W.parts > 1 ? (long long)A.G * N : A.ld_b;
  const long long all = (long long)A.B * A.T * A.G * N;
  float* dC = (W.parts > 1 ? W.part + 2 * part * all : A.dCm) + row0 * ldc + g * N;
  float* dB = (W.parts > 1 ? W.part + (2 * part + 1) * all : A.dBm) + row0 * ldb + g * N;

  if (here == 0) {  // padding: zeros
    for (int i = tid; i < rows * (N / 4); i += kThreads) {
      const int r = i / (N / 4), k = i % (N / 4) * 4;
      *(float4*)(dC + r * ldc + k) = make_float4(0.f, 0.f, 0.f, 0.f);
      *(float4*)(dB + r * ldb + k) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int h = h0; h < h1; ++h) {
      for (int i = tid; i < rows * (P / 4); i += kThreads)
        *(float4*)(A.dx + (row0 + i / (P / 4)) * A.ld_x + h * P + i % (P / 4) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tid < rows) A.ddt[(row0 + tid) * A.ld_dt + h] = 0.f;
      if (tid < 3) W.sums[(((long long)b * W.blocks + blk) * A.H + h) * 3 + tid] = 0.0;
    }
    return;
  }

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
  constexpr int E = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  // ---- B, C of the block and G = C B^T, tile t = wave + 7 e as [j][i]
  {
    constexpr int KR = NK * 32 / E, KN = (Q * KR + kThreads - 1) / kThreads;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
      const int q = tid + kThreads * i, j = q / KR, k = q % KR * E;
      if (j >= Q) break;
      const bool in = j < here && k < N;
      put(Bs, nB, j * LB + k, in ? *(const uint4*)((const char*)A.Bm + ((row0 + j) * A.ld_b + g * N + k) * ES) : zero, BF16);
      put(Cs, nB, j * LB + k, in ? *(const uint4*)((const char*)A.Cm + ((row0 + j) * A.ld_c + g * N + k) * ES) : zero, BF16);
    }
  }
  __syncthreads();
  // tiles per wave, the zero tiles behind the others; the last wave, which does the time steps, has none
  constexpr int MW = (MT + QT / 2 + kWaves - 2) / (kWaves - 1);
  const int tile0 = wave < kWaves - 1 ? wave : MT + QT / 2;
  int it_[MW], jt_[MW];
  f32x4_t G[MW];
#pragma unroll
  for (int e = 0; e < MW; ++e) {
    const int t = tile0 + (kWaves - 1) * e;
    int it = 1, jt = t - QT;
    while (jt >= it) jt -= it++;
    it_[e] = t < QT ? t : t < MT ? it : 2 * (t - MT);
    jt_[e] = t < QT ? t : t < MT ? jt : 2 * (t - MT) + 1;
    G[e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (t < MT) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
        mma(G[e], along<NP>(Bs + 16 * jt_[e] * LB + 32 * k, LB, nB, lane), along<NP>(Cs + 16 * it_[e] * LB + 32 * k, LB, nB, lane));
    }
  }

  // ---- tiles of the results: dx as [channel][token], channel tile pt, token tiles jx ..; dC and dB as
  // [d_k][token], d_k tile nt, token tiles ti ..
  constexpr int JW = QT / 2, TG = kWaves / NT > 1 ? kWaves / NT : 1, TW = QT / TG > 0 ? QT / TG : 1;
  const int pt = wave & 3, jx = (wave >> 2) * JW;
  const int nt = wave % NT, ti = wave / NT * TW;
  const bool owns = ti < QT;
  f32x4_t sC[TW], sB[TW];
#pragma unroll
  for (int r = 0; r < TW; ++r) sC[r] = sB[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  constexpr int XR = kPB / E, XN = (Q * XR + kThreads - 1) / kThreads, GR = kPB / 4, GN = (Q * GR + kThreads - 1) / kThreads;
  constexpr int UR = NK * 32 / 4, UN = kPB * UR / kThreads;
  uint4 rx[XN], rg[GN];
  auto fetch = [&](int h, int p0) {  // x and go of a head's channel block
    const rsrc_t rows_x = block_rows((const char*)A.x + (row0 * A.ld_x + h * P + p0) * ES, (uint32_t)(here * A.ld_x) * ES);
    const rsrc_t rows_g = block_rows(A.go + (((long long)b * A.H + h) * A.T + t0) * P + p0, (uint32_t)(here * P) * 4);
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int q = tid + kThreads * i, j = q / XR, k = q % XR * E;
      rx[i] = load16(rows_x, p0 + k < P ? (uint32_t)(j * A.ld_x + k) * ES : kNowhere);
    }
#pragma unroll
    for (int i = 0; i < GN; ++i) {
      const int q = tid + kThreads * i, j = q / GR, k = q % GR * 4;
      rg[i] = load16(rows_g, p0 + k < P ? (uint32_t)(j * P + k) * 4 : kNowhere);
    }
  };
  auto put_xg = [&] {
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int q = tid + kThreads * i, j = q / XR, k = q % XR * E;
      if (Q * XR % kThreads == 0 || j < Q) put(Xs, nX, j * LX + k, rx[i], BF16);
    }
#pragma unroll
    for (int i = 0; i < GN; ++i) {
      const int q = tid + kThreads * i, j = q / GR, k = q % GR * 4;
      if (Q * GR % kThreads == 0 || j < Q) put(Gs, nX, j * LX + k, rg[i], false);
    }
  };

  // the segments in which the two walks came to this block, and the blocks that those began with
  const int sseg = (int)(((long long)(blk + 1) * W.segments - 1) / W.blocks), seg_s = (int)((long long)W.blocks * sseg / W.segments);
  const int useg = (int)(((long long)(W.blocks - blk) * W.segments - 1) / W.blocks),
            seg_u = W.blocks - 1 - (int)((long long)W.blocks * useg / W.segments);
  auto joined = [](const uint4& v, const uint4& first, float upto) {
    return make_uint4(__float_as_uint(fmaf(__uint_as_float(first.x), upto, __uint_as_float(v.x))),
                      __float_as_uint(fmaf(__uint_as_float(first.y), upto, __uint_as_float(v.y))),
                      __float_as_uint(fmaf(__uint_as_float(first.z), upto, __uint_as_float(v.z))),
                      __float_as_uint(fmaf(__uint_as_float(first.w), upto, __uint_as_float(v.w))));
  };
  // Each tile of x and go is fetched as the one before it goes into LDS: of several channel blocks up for P,
  // down again for the rest, then the next head's first
  const int plast = (pblocks - 1) * kPB;
  fetch(h0, 0);
  double l_ahead;
  float step_ahead, dt_ahead;
  auto fetch_gates = [&](int h) {
    const long long gate = ((long long)b * A.H + h) * R.stride + t0 + (lane & (Q - 1));
    l_ahead = R.l[gate];
    step_ahead = R.step[gate];
    dt_ahead = A.dt[(row0 + min(lane, here - 1)) * A.ld_dt + h];
  };
  fetch_gates(h0);

  // ---- time steps of a head, one token per lane of a wave: the last one, beside the others' M and R of the next head
  int side = 0;  // where this head's sums go
  auto times = [&](int h, float step, float raw, double end) {
    anew();
    const int i = lane & (Q - 1), own = i / 16;
    double row = 0.0, col = 0.0, rd = 0.0, pu = 0.0, whole = 0.0;
#pragma unroll
    for (int u = 0; u < QT; ++u) {  // tiles of the token's row, and of its column
      const int lo = min(own, u), hi = max(own, u), t = lo == hi ? own : QT + hi * (hi - 1) / 2 + lo;
      const double a = row_[side ^ 1][t][i & 15], c = col_[side ^ 1][t][i & 15];
      row += u <= own ? a : 0.0;
      col += u >= own ? c : 0.0;
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      rd += (double)read_[k][i];
      pu += (double)put_[k][i];
    }
#pragma unroll
    for (int k = 0; k < kWaves; ++k) whole += us_[k];
    const bool in = lane < here;
    const float rate = -expf(A.A_log[h]);
    const double st = (double)step;
    const double ahead = in ? row - st * col + rd : 0.0, behind = in ? st * pu : 0.0;
    const double pa = block_prefix<64>(ahead), pp = block_prefix<64>(behind);
    const double dl = read_lane(pa, 63) - pa + ahead + pp - behind + (double)exp2_of(end) * whole;
    double ddt = 0.0, da = 0.0, tr = 0.0;
    if (in) {
      ddt = ((double)diag_[side ^ 1][i] + col + pu + dl * (double)rate) * (double)(1.f / (1.f + expf(-raw)));
      da = dl * (double)rate * st;
      tr = (double)trace_[side ^ 1][i];
    }
    if (lane < rows) A.ddt[(row0 + lane) * A.ld_dt + h] = (float)ddt;
    const double s0 = read_lane(block_prefix<64>(da), 63), s1 = read_lane(block_prefix<64>(ddt), 63),
                 s2 = read_lane(block_prefix<64>(tr), 63);
    if (lane < 3) W.sums[(((long long)b * W.blocks + blk) * A.H + h) * 3 + lane] = lane == 0 ? s0 : lane == 1 ? s1 : s2;
  };
  float step_before = 0.f, raw_before = 0.f;
  double end_before = 0.0;
  for (int h = h0; h < h1; ++h) {
    anew();
    const long long bh = (long long)b * A.H + h;
    const float D = A.D ? A.D[h] : 0.f;
    // S and U: what the segment adds (nothing before its first block), and of several segments what was before it
    const uint32_t state = (uint32_t)(P * N) * 4;
    const bool split = W.segments > 1;
    const int turned = turned_size(N, P);
    const rsrc_t rows_s = block_rows(W.S + (bh * W.blocks + blk) * turned, split && blk == seg_s ? 0u : (uint32_t)turned * 4);
    const rsrc_t rows_u = block_rows(W.U + (bh * W.blocks + blk) * P * N, split && blk == seg_u ? 0u : state);
    const rsrc_t rows_sf = block_rows(W.S_first + ((long long)sseg * A.B * A.H + bh) * turned, split ? (uint32_t)turned * 4 : 0u);
    const rsrc_t rows_uf = block_rows(W.U_first + ((long long)useg * A.B * A.H + bh) * P * N, split ? state : 0u);
    const float upto_s = split ? W.S_upto[bh * W.blocks + blk] : 0.f, upto_u = split ? W.U_upto[bh * W.blocks + blk] : 0.f;
    // ---- gates, by every wave in its lanes, one of them each into LDS
    const double l = l_ahead;
    const float step = step_ahead, raw = dt_ahead + A.dt_bias[h];
    const double end = read_lane(l, Q - 1);
    if (lane < Q) {
      if (wave == 0) l_[lane] = l;
      if (wave == 1) step_[lane] = step;
      if (wave == 2) since_[lane] = exp2_of(l);
      if (wave == 3) {
        const float w = exp2_of(end - l);
        w_[lane] = w;
        left_[lane] = w * step;
      }
    }
    double from = 0.0;
#pragma unroll
    for (int it = 1; it < QT; ++it) {
      const double at = read_lane(l, 16 * it - 1);
      from = lane >= 16 * it ? at : from;
    }
    if (wave == 7 && lane < Q) up_[lane] = exp2_of(l - from);

    // U of a channel block, fetched while the products before it run
    uint4 ru[UN], uf_[UN];
    auto fetch_u = [&](int p0) {
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int v = tid + kThreads * i, p = v / UR, k = v % UR * 4;
        const uint32_t at = p0 + p < P && k < N ? (uint32_t)((p0 + p) * N + k) * 4 : kNowhere;
        ru[i] = load16(rows_u, at);
        uf_[i] = load16(rows_uf, at);
      }
    };

    // ---- P = go x^T over the channel blocks; the last one's tiles stay
    f32x4_t Pm[MW];
#pragma unroll
    for (int e = 0; e < MW; ++e) Pm[e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int pb = 0; pb < pblocks; ++pb) {
      if (pb > 0) __syncthreads();  // the block before is read
      put_xg();
      if (pb + 1 < pblocks) fetch(h, (pb + 1) * kPB);
      else if (pblocks > 1) fetch(h, plast - kPB);
      else if (h + 1 < h1) fetch(h + 1, 0);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < MW; ++e)
        if (tile0 + (kWaves - 1) * e < MT) {
#pragma unroll
          for (int k = 0; k < kPB / 32; ++k)
            mma(Pm[e], along<NP>(Xs + 16 * jt_[e] * LX + 32 * k, LX, nX, lane), along<3>(Gs + 16 * it_[e] * LX + 32 * k, LX, nX, lane));
        }
    }

    fetch_gates(min(h + 1, h1 - 1));
    if (wave == kWaves - 1 && h > h0) times(h - 1, step_before, raw_before, end_before);
    anew();
    // ---- M and R (R's columns in the order of across()), sums over rows and columns of F
#pragma unroll
    for (int e = 0; e < MW; ++e) {
      const int t = tile0 + (kWaves - 1) * e;
      if (t >= MT + QT / 2) break;
      const int i = 16 * it_[e] + lr, j = 16 * jt_[e] + 4 * lg;
      float m[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
      if (t < MT) {
        const bool diag = t < QT;
        const f32x4_t st = *(const f32x4_t*)(step_ + j);
        double row = 0.0, col[4];
        float dec[4];  // E
        if (diag) {
          const double li = l_[i];
          const double2 a0 = *(const double2*)(l_ + j), a1 = *(const double2*)(l_ + j + 2);
          const double lj[4] = {a0.x, a0.y, a1.x, a1.y};
#pragma unroll
          for (int u = 0; u < 4; ++u) dec[u] = exp2_of(li - lj[u]);
        } else {
          // over the start of the row's tile: both factors are at most 1
          const double at = l_[16 * it_[e] - 1];
          const double2 a0 = *(const double2*)(l_ + j), a1 = *(const double2*)(l_ + j + 2);
          const double lj[4] = {a0.x, a0.y, a1.x, a1.y};
          const float up = up_[i];
#pragma unroll
          for (int u = 0; u < 4; ++u) dec[u] = up * exp2_of(at - lj[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t keep = !diag || j + u <= i ? ~0u : 0u, self = diag && j + u == i ? ~0u : 0u;
          const float ge = __uint_as_float(__float_as_uint(G[e][u] * dec[u]) & keep);
          const float pe = __uint_as_float(__float_as_uint(Pm[e][u] * dec[u]) & keep);
          const float f = __uint_as_float(__float_as_uint(Pm[e][u] * ge) & keep);
          m[u] = ge * st[u] + __uint_as_float(__float_as_uint(D) & self);
          r[u] = pe * st[u];
          if (self) {
            diag_[side][i] = f;
            trace_[side][i] = Pm[e][u];
          }
          const double off = (double)__uint_as_float(__float_as_uint(f) & ~self);
          col[u] = off;
          row += off * (double)st[u];
        }
        // over the columns: the four groups of 16 lanes; over the rows: the lanes of a group
        row += __shfl_xor(row, 16, 64);
        row += __shfl_xor(row, 32, 64);
        if (lg == 0) row_[side][t][lr] = row;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          double v = col[u];
          v = add_dpp<0x111, 0xF>(v);
          v = add_dpp<0x112, 0xF>(v);
          v = add_dpp<0x114, 0xF>(v);
          v = add_dpp<0x118, 0xF>(v);
          if (lr == 15) col_[side][t][4 * lg + u] = v;
        }
      }
      uint32_t a[3], d[3];
      split_pair(m[0], m[1], a);
      split_pair(m[2], m[3], d);
#pragma unroll
      for (int k = 0; k < 3; ++k) *(uint2*)(Ms + k * nM + i * LM + j) = make_uint2(a[k], d[k]);
      split_pair(r[0], r[1], a);
      split_pair(r[2], r[3], d);
#pragma unroll
      for (int k = 0; k < 3; ++k) *(uint2*)(Rs + k * nM + i * LM + across_order(j)) = make_uint2(a[k], d[k]);
    }
    __syncthreads();

    anew();
    // ---- inside the block: dC, dB; dx of every channel block, the one in LDS first
    if (owns) {
#pragma unroll
      for (int r = 0; r < TW; ++r) {
        const int t = ti + r;
#pragma unroll
        for (int k = 0; k < Q / 32; ++k) {
          if (k <= t / 2) mma(sC[r], across<NP>(Bs + 32 * k * LB + 16 * nt, LB, nB, lane), along<3>(Rs + 16 * t * LM + 32 * k, LM, nM, lane));
          if (k >= t / 2)
            mma(sB[r], across<NP>(Cs + 32 * k * LB + 16 * nt, LB, nB, lane),
                across<3, 8>(Rs + 32 * k * LM + 32 * (t >> 1) + 4 * (t & 1), LM, nM, lane));
        }
      }
    }
    fetch_u(plast);
    f32x4_t T1[TW], T2[TW];
#pragma unroll
    for (int r = 0; r < TW; ++r) T1[r] = T2[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    double us = 0.0;
    for (int q = 0; q < pblocks; ++q) {
      const int pb = pblocks - 1 - q, p0 = pb * kPB;
      anew();
      f32x4_t dx[JW], du[JW];
#pragma unroll
      for (int r = 0; r < JW; ++r) dx[r] = du[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (q > 0) {
        // (several channel blocks) M's place holds U of the block before: form it again from the registers
        __syncthreads();
        put_xg();
        if (pb > 0) fetch(h, p0 - kPB);
        else if (h + 1 < h1) fetch(h + 1, 0);
#pragma unroll
        for (int e = 0; e < MW; ++e) {
          const int t = tile0 + (kWaves - 1) * e;
          if (t >= MT + QT / 2) break;
          const int i = 16 * it_[e] + lr, j = 16 * jt_[e] + 4 * lg;
          float m[4] = {0.f, 0.f, 0.f, 0.f};
          if (t < MT) {
            const bool diag = t < QT;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const double at = diag ? l_[i] : l_[16 * it_[e] - 1];
              const float dec = exp2_of(at - l_[j + u]) * (diag ? 1.f : up_[i]);
              const uint32_t keep = !diag || j + u <= i ? ~0u : 0u, self = diag && j + u == i ? ~0u : 0u;
              const float ge = __uint_as_float(__float_as_uint(G[e][u] * dec) & keep);
              m[u] = ge * step_[j + u] + __uint_as_float(__float_as_uint(D) & self);
            }
          }
          uint32_t a[3], d[3];
          split_pair(m[0], m[1], a);
          split_pair(m[2], m[3], d);
#pragma unroll
          for (int k = 0; k < 3; ++k) *(uint2*)(Ms + k * nM + i * LM + j) = make_uint2(a[k], d[k]);
        }
        __syncthreads();
      }
      // S^T for the state's share: d_k of this lane, 8 channels a step
      uint4 rs[kPB / 32][2], sf_[kPB / 32][2];
#pragma unroll
      for (int k = 0; k < kPB / 32; ++k) {
        const int p = p0 + 32 * k + 8 * lg, kk = 16 * nt + lr;
        const uint32_t at = p < P && kk < N ? (uint32_t)turned_at(nt, P, p, lr) * 4 : kNowhere;
        rs[k][0] = load16(rows_s, at);
        rs[k][1] = load16(rows_s, at + 1024);
        sf_[k][0] = load16(rows_sf, at);
        sf_[k][1] = load16(rows_sf, at + 1024);
      }
#pragma unroll
      for (int r = 0; r < JW; ++r)
#pragma unroll
        for (int k = 0; k < Q / 32; ++k)
          if (k >= (jx + r) / 2)
            mma(dx[r], across<3, 8>(Gs + 32 * k * LX + 32 * (pt >> 1) + 4 * (pt & 1), LX, nX, lane),
                across<3>(Ms + 32 * k * LM + 16 * (jx + r), LM, nM, lane));
      __syncthreads();  // M and R are read
      // (U's rows in the order in which across() takes them)
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int v = tid + kThreads * i, p = v / UR, k = v % UR * 4;
        const int at = (p & 32) | ((p & 4) << 2) | ((p & 24) >> 1) | (p & 3);
        put(Us, nU, at * LU + k, joined(ru[i], uf_[i], upto_u), false);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const Frag<3> uf = along<3>(Us + 16 * pt * LU + 32 * k, LU, nU, lane);
#pragma unroll
        for (int r = 0; r < JW; ++r) mma(du[r], uf, along<NP>(Bs + 16 * (jx + r) * LB + 32 * k, LB, nB, lane));
      }
      if (owns) {
#pragma unroll
        for (int k = 0; k < kPB / 32; ++k) {
          const uint4 s0 = joined(rs[k][0], sf_[k][0], upto_s), s1 = joined(rs[k][1], sf_[k][1], upto_s);
          const float sv[8] = {__uint_as_float(s0.x), __uint_as_float(s0.y), __uint_as_float(s0.z), __uint_as_float(s0.w),
                               __uint_as_float(s1.x), __uint_as_float(s1.y), __uint_as_float(s1.z), __uint_as_float(s1.w)};
          const Frag<3> sf = split8(sv), uf = across<3>(Us + 32 * k * LU + 16 * nt, LU, nU, lane);
          if (wave < NT) {
            float uv[8];
            values_of(uf, uv);
#pragma unroll
            for (int v = 0; v < 8; ++v) us += (double)(uv[v] * sv[v]);
          }
#pragma unroll
          for (int r = 0; r < TW; ++r) {
            mma(T1[r], sf, along<3>(Gs + 16 * (ti + r) * LX + 32 * k, LX, nX, lane));
            mma(T2[r], uf, along<NP>(Xs + 16 * (ti + r) * LX + 32 * k, LX, nX, lane));
          }
        }
      }
      if (pb > 0) fetch_u(p0 - kPB);
      const int pp = p0 + 32 * (pt >> 1) + 8 * lg + 4 * (pt & 1);
#pragma unroll
      for (int r = 0; r < JW; ++r) {
        const int j = 16 * (jx + r) + lr;
        if (j < rows && pp < P)
          *(f32x4_t*)(A.dx + (row0 + j) * A.ld_x + h * P + pp) = j < here ? dx[r] + du[r] * left_[j] : f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
    anew();
    // ---- the states' shares of dC and dB, and of the decays' gradients
    if (owns) {
#pragma unroll
      for (int r = 0; r < TW; ++r) {
        const int i = 16 * (ti + r) + lr;
        const f32x4_t c1 = T1[r] * since_[i];
        sC[r] += c1;
        sB[r] += T2[r] * left_[i];
        float cd = 0.f, bd = 0.f;
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) {
          const uint2 cv = *(const uint2*)(Cs + k * nB + i * LB + 16 * nt + 4 * lg), bv = *(const uint2*)(Bs + k * nB + i * LB + 16 * nt + 4 * lg);
          cd += c1[0] * bf16lo(cv.x) + c1[1] * bf16hi(cv.x) + c1[2] * bf16lo(cv.y) + c1[3] * bf16hi(cv.y);
          bd += T2[r][0] * bf16lo(bv.x) + T2[r][1] * bf16hi(bv.x) + T2[r][2] * bf16lo(bv.y) + T2[r][3] * bf16hi(bv.y);
        }
        cd = add_xor_f32(add_xor_f32(cd, 16), 32);
        bd = add_xor_f32(add_xor_f32(bd, 16), 32);
        if (lg == 0) {
          read_[nt][i] = cd;
          put_[nt][i] = bd * w_[i];
        }
      }
    }
    us = block_prefix<64>(us);
    if (lane == 63) us_[wave] = us;
    __syncthreads();

    step_before = step;
    raw_before = raw;
    end_before = end;
    side ^= 1;
  }
  if (wave == kWaves - 1) times(h1 - 1, step_before, raw_before, end_before);

  if (owns) {
    const int k = 16 * nt + 4 * lg;
#pragma unroll
    for (int r = 0; r < TW; ++r) {
      const int i = 16 * (ti + r) + lr;
      if (i < rows && k < N) {
        *(f32x4_t*)(dC + i * ldc + k) = i < here ? sC[r] : f32x4_t{0.f, 0.f, 0.f, 0.f};
        *(f32x4_t*)(dB + i * ldb + k) = i < here ? sB[r] : f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
}

// Workgroups 0 .. H-1: a head's sums over sequences and blocks. The others: dC and dB from the parts of a
// group's heads. All in their order.
__global__ void __launch_bounds__(256) scan_finish_kernel(ScanArgs A, ScanBwd W) {
  if ((int)blockIdx.x < A.H) {
    __shared__ double part[4][3];
    const int h = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double s[3] = {};
    for (long long i = threadIdx.x; i < (long long)A.B * W.blocks; i += 256)
      for (int k = 0; k < 3; ++k) s[k] += W.sums[(i * A.H + h) * 3 + k];
    for (int k = 0; k < 3; ++k) {
      s[k] = block_prefix<64>(s[k]);
      if (lane == 63) part[wave][k] = s[k];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int k = 0; k < 3; ++k) s[k] = (part[0][k] + part[1][k]) + (part[2][k] + part[3][k]);
      A.dA_log[h] = (float)s[0];
      A.ddt_bias[h] = (float)s[1];
      if (A.dD) A.dD[h] = (float)s[2];
    }
    return;
  }
  const int per = A.G * A.N / 4;
  const long long tokens = (long long)A.B * A.T, i = (long long)(blockIdx.x - A.H) * 256 + threadIdx.x;
  if (i >= 2 * tokens * per) return;
  const int what = (int)(i / (tokens * per));
  const long long at = i % (tokens * per), row = at / per;
  const int k = (int)(at % per) * 4;
  const f32x4_t* v = (const f32x4_t*)W.part + what * tokens * per + at;
  f32x4_t s = v[0];
  for (int p = 1; p < W.parts; ++p) s += v[2 * p * tokens * per];
  *(f32x4_t*)((what ? A.dBm + row * A.ld_b : A.dCm + row * A.ld_c) + k) = s;
}

struct BwdPlan {
  ScanGates gates;
  ScanBwd bwd;
  double *decay, *decay_back;
  size_t bytes;
};

// A group's heads are shared out over workgroups, one of which fills a compute unit: for the fewest rounds of
// 256 times a workgroup's length, in which the products of B and C count as half a head.
BwdPlan plan_of(const sdm_scan_shape& S, char* base) {
  BwdPlan L{};
  const int Q = S.in_dtype == SDM_BF16 ? 64 : 32, hpg = S.H / S.G;
  const size_t units = (size_t)S.B * S.H, state = (size_t)S.d_v * S.d_k * 4, turned = (size_t)turned_size(S.d_k, S.d_v) * 4;
  L.bwd.blocks = (S.T + Q - 1) / Q;
  const long long groups = (long long)S.B * S.G * L.bwd.blocks;
  long long parts = 1;
  double best = 0.0;
  for (int p = 1; p <= hpg && p <= 512; ++p) {
    const double cost = (double)((groups * p + 255) / 256) * ((hpg + p - 1) / p + 0.5);
    if (p == 1 || cost < best) {
      parts = p;
      best = cost;
    }
  }
  L.bwd.heads = (int)((hpg + parts - 1) / parts);
  L.bwd.parts = (hpg + L.bwd.heads - 1) / L.bwd.heads;
  // (each walk in 256 workgroups, as two fit a compute unit: three times as many, whose first states the blocks
  // then read more of, took 175 us instead of 162 at 4 x 2048 tokens, 8 heads of 128 x 128)
  L.bwd.segments = scan_segments((long long)units * ((S.d_v + kPB - 1) / kPB), L.bwd.blocks, 256);
  size_t at = gates_bytes(units, S.T, base, &L.gates);
  L.bwd.S = (float*)(base + at);
  at += align_up(units * L.bwd.blocks * turned);
  L.bwd.U = (float*)(base + at);
  at += align_up(units * L.bwd.blocks * state);
  L.bwd.sums = (double*)(base + at);
  at += align_up((size_t)S.B * L.bwd.blocks * S.H * 24);
  if (L.bwd.parts > 1) {
    L.bwd.part = (float*)(base + at);
    at += align_up((size_t)L.bwd.parts * 2 * S.B * S.T * S.G * S.d_k * 4);
  }
  if (L.bwd.segments > 1) {
    const size_t slots = units * (L.bwd.segments + 1), factors = align_up(units * L.bwd.blocks * 4);
    L.bwd.S_first = (float*)(base + at);
    at += align_up(slots * turned);
    L.bwd.U_first = (float*)(base + at);
    at += align_up(slots * state);
    L.decay = (double*)(base + at);
    L.decay_back = (double*)(base + at + align_up(slots * 8));
    at += 2 * align_up(slots * 8);
    L.bwd.S_upto = (float*)(base + at);
    L.bwd.U_upto = (float*)(base + at + factors);
    at += 2 * factors;
  }
  L.bytes = at + 256;  // (never empty)
  return L;
}

template <bool BF16, int NK>
hipError_t launch_main(const ScanArgs& A, const BwdPlan& L, hipStream_t stream) {
  constexpr int lds = BwdTiles<BF16, NK>::bytes;
  const long long grid = (long long)A.B * A.G * L.bwd.blocks * L.bwd.parts;
  hipLaunchKernelGGL((scan_backward_kernel<BF16, NK>), dim3((unsigned)grid), dim3(kThreads), lds, stream, A, L.gates, L.bwd);
  return hipGetLastError();
}

}  // namespace

size_t scan_backward_workspace_bytes(const sdm_scan_shape& S) { return plan_of(S, nullptr).bytes; }

hipError_t launch_scan_backward(const sdm_scan_shape& S, const ScanArgs& A, hipStream_t stream) {
  const BwdPlan L = plan_of(S, (char*)A.ws);
  hipError_t e = launch_scan_gates(A, A.bf16 ? 64 : 32, L.gates, stream);
  if (e != hipSuccess) return e;
  ScanWalk K{};
  K.B = A.B;
  K.T = A.T;
  K.H = A.H;
  K.G = A.G;
  K.N = A.N;
  K.P = A.P;
  K.blocks = L.bwd.blocks;
  K.segments = L.bwd.segments;
  K.stride = L.gates.stride;
  K.lengths = A.lengths;
  K.l = L.gates.l;
  K.first = (float*)L.bwd.S_first;
  K.upto = (float*)L.bwd.S_upto;
  K.decay = L.decay;
  K.X = A.x;
  K.K = A.Bm;
  K.xb = (long long)A.T * A.ld_x;
  K.xh = A.P;
  K.ld_x = A.ld_x;
  K.ld_k = A.ld_b;
  K.weight = L.gates.left;
  K.start = A.s_in;
  K.states = (float*)L.bwd.S;
  ScanWalk U = K;  // and back, for the states' gradients
  U.X = A.go;
  U.K = A.Cm;
  U.xb = (long long)A.H * A.T * A.P;
  U.xh = (long long)A.T * A.P;
  U.ld_x = A.P;
  U.ld_k = A.ld_c;
  U.weight = L.gates.since;
  U.start = A.ds_out;
  U.end = A.ds_in;
  U.states = (float*)L.bwd.U;
  U.first = (float*)L.bwd.U_first;
  U.decay = L.decay_back;
  U.upto = (float*)L.bwd.U_upto;
  e = launch_scan_walks(K, U, A.bf16, stream);
  if (e != hipSuccess) return e;
  if (L.bwd.blocks > 0) {
    e = A.bf16   ? (A.N <= 32   ? launch_main<true, 1>(A, L, stream)
                    : A.N <= 64 ? launch_main<true, 2>(A, L, stream)
                                : launch_main<true, 4>(A, L, stream))
        : A.N <= 32 ? launch_main<false, 1>(A, L, stream)
        : A.N <= 64 ? launch_main<false, 2>(A, L, stream)
                    : launch_main<false, 4>(A, L, stream);
    if (e != hipSuccess) return e;
  }
  const long long quads = L.bwd.blocks > 0 && L.bwd.parts > 1 ? 2ll * A.B * A.T * (A.G * A.N / 4) : 0;
  hipLaunchKernelGGL(scan_finish_kernel, dim3((unsigned)(A.H + (quads + 255) / 256)), dim3(256), 0, stream, A, L.bwd);
  return hipGetLastError();
}

}  // namespace sdm
