// Selective state space scan: a dense state per head that decays by a scalar of the token and takes
// up an outer product of the token's channels and its B, read through its C.
//
//   dtv = softplus(dt + dt_bias), a = exp(-exp(A_log) dtv)
//   S_t = a_t S_{t-1} + dtv_t x_t B_t^T,   o_t = S_t C_t + D x_t
//
// Prompts run in blocks of Q tokens. With l the log-decay summed from the block's start, S the state
// before the block and M_ij = (C_i . B_j) exp(l_i - l_j) dtv_j for j <= i, D more for j = i:
//   o_i = exp(l_i) S C_i + sum_j M_ij x_j
//   S'  = exp(l_end) S + sum_j (exp(l_end - l_j) dtv_j x_j) B_j^T
// all of them matrix products. l is summed in float64, so that the differences keep their digits.
//
// Float32 factors go into the matrix products as three bf16 pieces each, whose products are as exact as
// float32's, at 3 (beside a bf16 factor) or 6 times a bf16 product's work. That work bounds prompts, not memory: at 131072 tokens, 8 heads of 128 x 128, 370 GFLOP,
// 310 us at the rate of a large bf16 product and 190 us of memory traffic. Measured 542 us (this kernel 390-470,
// the walk 150, gates 13, join 11); 8 x 4096 tokens, 16 heads of 128 x 64: 149 us (104, 38, 9, 7). A wave's vector
// work (splitting, decays) takes as long as its matrix work and two waves per SIMD, all that registers and LDS
// hold, do not overlap the two wholly.

#include "sdm_device.hpp"
#include "sdm_internal.hpp"
#include "sdm_scan.hpp"

namespace sdm {

namespace {

constexpr int kPB = 64;  // channels per workgroup: 16 for each of its 4 waves

// Tokens per block: the tiles of three pieces of float32 inputs fill LDS at half the bf16 block
template <bool BF16>
constexpr int block_tokens() { return BF16 ? 64 : 32; }

struct ScanPlan {
  int pblocks;   // channel blocks per head
  int blocks;    // token blocks
  int segments;  // token segments
};

struct ScanWs {
  float* first;   // [segments][B*H][P][N]: states before the segments
  double* decay;  // [segments][B*H]: log2 of the segments' decay
};

// LDS of one workgroup: tiles of B, x, C (NP planes each) and M (3 planes). Row strides keep the 8-byte
// reads along rows and the transposing reads over 16 rows on different banks.
template <bool BF16, int NK>
struct Tiles {
  static constexpr int Q = block_tokens<BF16>(), NP = BF16 ? 1 : 3;
  static constexpr int LB = NK * 32 + 16, LC = NK * 32 + 8, LX = kPB + 16, LM = Q + 8;
  static constexpr int nB = Q * LB, nC = Q * LC, nX = Q * LX, nM = Q * LM;
  static constexpr int bytes = (NP * (nB + nX + nC) + 3 * nM) * 2;
};

// ------------------------------------------------------------------ prompts
// One workgroup walks the blocks of a segment of a (sequence, head, 64 channels) unit with the state in
// the accumulators of its matrix products: wave w holds channels 16 w .. 16 w + 15, all d_k. So the state is
// never stored between blocks, and each wave splits its own part of it only. Blocks of 64 tokens: the state's
// products are shared by more tokens than in smaller ones, M grows with their square.
template <bool BF16, int NK>
__global__ void __launch_bounds__(256, 2) scan_kernel(ScanArgs A, ScanPlan L, ScanWs W, ScanGates R) {
  using TL = Tiles<BF16, NK>;
  constexpr int Q = TL::Q, NP = TL::NP, NT = 2 * NK, QT = Q / 16;
  constexpr int LB = TL::LB, LC = TL::LC, LX = TL::LX, LM = TL::LM, nB = TL::nB, nC = TL::nC, nX = TL::nX, nM = TL::nM;
  extern __shared__ __align__(16) uint16_t lds[];
  // of the block: log-decays, steps, factors to the token and to the block's end, and for the tiles of M off
  // the diagonal the factors from the start of a token's tile to it and from a token to the start of tile it
  __shared__ __align__(16) double l_[Q];
  __shared__ __align__(16) float step_[Q], since_[Q], left_[Q], up_[Q], down_[QT][Q];
  __shared__ int bad_[2];  // does x of the block hold an infinity or a NaN, by the block's parity
  uint16_t *Bs = lds, *Xs = Bs + NP * nB, *Cs = Xs + NP * nX, *Ms = Cs + NP * nC;

  // unit: the heads of a group side by side on one XCD (workgroups go to the 8 XCDs in turn), so that its
  // L2 holds the B and C they share
  const int hpg = A.H / A.G;
  const int fast = A.B * A.G * L.segments;
  const int f = blockIdx.x % fast, s = blockIdx.x / fast;
  const int seg = f / (A.B * A.G), bg = f % (A.B * A.G), b = bg / A.G, g = bg % A.G;
  const int h = g * hpg + s % hpg, pb = s / hpg;
  const long long bh = (long long)b * A.H + h;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lg = lane >> 4, lr = lane & 15;
  const int n = sequence_length(A.lengths, b, A.T);
  const int N = A.N, P = A.P, p0 = pb * kPB;
  const int c0 = (int)((long long)L.blocks * seg / L.segments), c1 = (int)((long long)L.blocks * (seg + 1) / L.segments);
  const float D = A.D ? A.D[h] : 0.f;

  // 16-byte pieces of a block's tiles: piece i of this thread lies in row j + i (256 / pieces-per-row) for
  // its row j of piece 0, in the same columns
  constexpr int E = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;        // values per piece, bytes per value
  constexpr int XR = kPB / E, KR = NK * 32 / E;             // pieces per row
  constexpr int NX = Q * XR / 256, NKV = (Q * KR + 255) / 256;      // pieces per thread
  constexpr int XS = 256 / XR, KS = 256 / KR;               // rows between pieces
  const int xj = tid / XR, xk = (tid % XR) * E, kj = tid / KR, kk = (tid % KR) * E;
  const uint32_t xoff = p0 + xk < P ? (uint32_t)(xj * A.ld_x + xk) * ES : kNowhere,
                 boff = kk < N ? (uint32_t)(kj * A.ld_b + kk) * ES : kNowhere,
                 coff = kk < N ? (uint32_t)(kj * A.ld_c + kk) * ES : kNowhere;
  const uint32_t xstep = (uint32_t)(XS * A.ld_x) * ES, bstep = (uint32_t)(KS * A.ld_b) * ES,
                 cstep = (uint32_t)(KS * A.ld_c) * ES;
  uint4 rx[NX], rb[NKV], rc[NKV];
  // the next block's rows, on by a block after each fetch
  const long long row0 = (long long)b * A.T + (long long)c0 * Q;
  const char* px = (const char*)A.x + (row0 * A.ld_x + h * P + p0) * ES;
  const char* pB = (const char*)A.Bm + (row0 * A.ld_b + g * N) * ES;
  const char* pC = (const char*)A.Cm + (row0 * A.ld_c + g * N) * ES;
  const long long xblock = Q * A.ld_x * ES, bblock = Q * A.ld_b * ES, cblock = Q * A.ld_c * ES;
  auto advance = [&] {
    px += xblock;
    pB += bblock;
    pC += cblock;
  };
  // part `part` of `parts` of a block's pieces, `here` of its tokens inside the sequence
  auto fetch = [&](int here, int part, int parts) {
    const rsrc_t rows_x = block_rows(px, (uint32_t)(here * A.ld_x) * ES), rows_b = block_rows(pB, (uint32_t)(here * A.ld_b) * ES),
                 rows_c = block_rows(pC, (uint32_t)(here * A.ld_c) * ES);
#pragma unroll
    for (int i = 0; i < NKV; ++i)
      if (i % parts == part) {
        rb[i] = load16(rows_b, boff + i * bstep);
        rc[i] = load16(rows_c, coff + i * cstep);
      }
#pragma unroll
    for (int i = 0; i < NX; ++i)
      if (i % parts == part) rx[i] = load16(rows_x, xoff + i * xstep);
  };
  // the block's gates, one token per lane
  double rl = 0.0;
  float rstep = 0.f, rfac = 0.f;
  const long long gate0 = bh * R.stride + (long long)c0 * Q;
  const double* gl = R.l + gate0;
  const float *gstep = R.step + gate0, *gfac = (wave == 2 ? R.since : R.left) + gate0;
  auto fetch_gates = [&](int on) {  // `on` tokens further than the last time
    gl += on;
    gstep += on;
    gfac += on;
    const int at = lane & (Q - 1);
    rl = gl[at];
    rstep = gstep[at];
    rfac = gfac[at];
  };
  auto put_gates = [&] {
    if (lane < Q) {
      if (wave == 3) left_[lane] = rfac;
      if (wave == 0) l_[lane] = rl;
      if (wave == 1) step_[lane] = rstep;
      if (wave == 2) since_[lane] = rfac;
    }
    double from = 0.0;  // log-decay at the start of this lane's tile
#pragma unroll
    for (int it = 1; it < QT; ++it) {
      const double at = read_lane(rl, 16 * it - 1);
      from = lane >= 16 * it ? at : from;
      if (wave == it && lane < 16 * it) down_[it][lane] = exp2_of(at - rl) * rstep;
    }
    if (wave == 0 && lane < Q) up_[lane] = exp2_of(rl - from);
  };
  // a piece into its tile: as it is, or its four float32 values as three bf16 planes
  auto put = [&](uint16_t* tile, int plane, int at, const uint4& v) {
    if (BF16) {
      *(uint4*)(tile + at) = v;
    } else {
      uint32_t a[3], d[3];
      split_pair(__uint_as_float(v.x), __uint_as_float(v.y), a);
      split_pair(__uint_as_float(v.z), __uint_as_float(v.w), d);
#pragma unroll
      for (int k = 0; k < 3; ++k) *(uint2*)(tile + k * plane + at) = make_uint2(a[k], d[k]);
    }
  };
  // the largest exponents of a piece's values, by halves (bf16) or in the high half: 0x7F80 and more in
  // infinities and NaNs
  auto exponents = [&](u16x2_t m, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu));
    return m;
  };

  // state: tiles of 16 d_k x 16 channels, in pairs over 32 d_k: this lane holds channel p0 + 16 wave + lr,
  // d_k 32 (m / 2) + 8 lg + 4 (m % 2) + 0..3 of tile m
  const int p = p0 + 16 * wave + lr;
  auto state_at = [&](int m) { return 32 * (m >> 1) + 8 * lg + 4 * (m & 1); };
  const long long srow = (bh * P + p) * N;
  f32x4_t S[NT];
  {
    const float* from = L.segments > 1 ? W.first + (long long)seg * A.B * A.H * P * N : A.s_in;
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int k = state_at(m);
      S[m] = from && p < P && k < N ? *(const f32x4_t*)(from + srow + k) : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }

  // the tiles of M right of the diagonal stay 0
  for (int i = tid; i < 3 * nM / 8; i += 256) ((uint4*)Ms)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) bad_[c0 & 1] = 0;
  if (c0 < c1) fetch_gates(0);
  fetch(min(max(n - c0 * Q, 0), Q), 0, 1);
  advance();
  float* orow = A.o + (bh * A.T + (long long)c0 * Q) * P;
  const uint32_t ooff = p0 + 16 * wave + 4 * lg < P ? (uint32_t)(lr * P + p0 + 16 * wave + 4 * lg) * 4 : kNowhere;
  for (int c = c0; c < c1; ++c, orow += Q * P) {
    const int left = n - c * Q, here = min(max(left, 0), Q), next = c + 1 < c1 ? min(max(left - Q, 0), Q) : 0, rows = min(A.T - c * Q, Q);
    if (here == 0) {  // behind the sequence's end, like every block after it
        for (int i = tid; i < rows * (kPB / 4); i += 256) {
          const int k = (i % (kPB / 4)) * 4;
          if (p0 + k < P) *(float4*)(orow + (long long)(i / (kPB / 4)) * P + p0 + k) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      continue;
    }
    __syncthreads();  // the tiles of the block before are read
    u16x2_t most = {0, 0};
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      put(Xs, nX, (xj + i * XS) * LX + xk, rx[i]);
      most = exponents(most, rx[i]);
    }
#pragma unroll
    for (int i = 0; i < NKV; ++i) {
      if (Q * KR % 256 != 0 && kj + i * KS >= Q) continue;
      put(Bs, nB, (kj + i * KS) * LB + kk, rb[i]);
      put(Cs, nC, (kj + i * KS) * LC + kk, rc[i]);
    }
    if ((most[1] >= 0x7F80 || (BF16 && most[0] >= 0x7F80))) bad_[c & 1] = 1;
    put_gates();
    const double end = read_lane(rl, Q - 1);
    fetch_gates(c + 1 < c1 ? Q : 0);
    __syncthreads();
    // x of this wave's channels, tokens along k; and weighted for the state at the block's end
    const float keep = exp2_of(end);
    Frag<NP> xf[Q / 32];
    Frag<3> xw[Q / 32];
    auto load_x = [&] {
#pragma unroll
      for (int k = 0; k < Q / 32; ++k) xf[k] = across<NP>(Xs + 32 * k * LX + 16 * wave, LX, nX, lane);
    };
    auto weigh_x = [&](int k) {
      float v[8];
      values_of(xf[k], v);
      const float4 w0 = *(const float4*)(left_ + 32 * k + 4 * lg), w1 = *(const float4*)(left_ + 32 * k + 16 + 4 * lg);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] *= w[u];
      xw[k] = split8(v);
    };

    if (tid == 0) bad_[(c + 1) & 1] = 0;
    // M, tiles (it, jt) in turn over the waves, those on the diagonal first; a wave without one more
    // repeats the last
    constexpr int MT = QT * (QT + 1) / 2, MW = (MT + 3) / 4;
    f32x4_t G[MW];
    int it_[MW], jt_[MW];
#pragma unroll
    for (int e = 0; e < MW; ++e) {
      const int t = min(wave + 4 * e, MT - 1);
      int it = 1, jt = t - QT;
      while (jt >= it) jt -= it++;
      it_[e] = t < QT ? t : it;
      jt_[e] = t < QT ? t : jt;
      G[e] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    Frag<NP> gb[2][MW], gc[2][MW];
    auto load_g = [&](int k) {
#pragma unroll
      for (int e = 0; e < MW; ++e) {
        gb[k & 1][e] = along<NP>(Bs + 16 * jt_[e] * LB + 32 * k, LB, nB, lane);
        gc[k & 1][e] = along<NP>(Cs + 16 * it_[e] * LC + 32 * k, LC, nC, lane);
      }
    };
    load_g(0);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k + 1 < NK) load_g(k + 1);
      stage();
#pragma unroll
      for (int e = 0; e < MW; ++e) mma(G[e], gb[k & 1][e], gc[k & 1][e]);
    }
    auto put_m = [&](int e) {  // tile e of this wave: decays, steps, three pieces
      const int i = 16 * it_[e] + lr, j = 16 * jt_[e] + 4 * lg;
      float mv[4];
      // (four token tiles: every wave's first is on the diagonal, its others are not)
      const bool diagonal = QT == 4 ? e == 0 : it_[e] == jt_[e];
      if (!diagonal) {
        const float up = up_[i];
        const f32x4_t down = *(const f32x4_t*)(down_[it_[e]] + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) mv[u] = G[e][u] * (up * down[u]);
      } else {
        const double li = l_[i];
        const double2 l0 = *(const double2*)(l_ + j), l1 = *(const double2*)(l_ + j + 2);
        const f32x4_t step = *(const f32x4_t*)(step_ + j);
        const double lj[4] = {l0.x, l0.y, l1.x, l1.y};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // right of the diagonal whatever the product is gives 0, by its bits: no branch around the exp
          const float v = G[e][u] * (exp2_of(li - lj[u]) * step[u]);
          mv[u] = __uint_as_float(__float_as_uint(v) & (j + u <= i ? ~0u : 0u)) +
                  __uint_as_float(__float_as_uint(D) & (j + u == i ? ~0u : 0u));
        }
      }
      uint32_t w0[3], w1[3];
      split_pair(mv[0], mv[1], w0);
      split_pair(mv[2], mv[3], w1);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *(uint2*)(Ms + k * nM + i * LM + across_order(j)) = make_uint2(w0[k], w1[k]);
    };
    f32x4_t Y[QT];
    Frag<NP> cf[2][QT];
    auto load_c = [&](int k) {
#pragma unroll
      for (int it = 0; it < QT; ++it) cf[k & 1][it] = along<NP>(Cs + 16 * it * LC + 32 * k, LC, nC, lane);
    };
    load_c(0);
#pragma unroll
    for (int it = 0; it < QT; ++it) Y[it] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    Frag<3> Sf[2];
    auto split_s = [&](int k) {  // the pieces of 32 d_k of the state, which then decays to the block's end
      const float v[8] = {S[2 * k][0], S[2 * k][1], S[2 * k][2], S[2 * k][3],
                          S[2 * k + 1][0], S[2 * k + 1][1], S[2 * k + 1][2], S[2 * k + 1][3]};
      Sf[k & 1] = split8(v);
      S[2 * k] *= keep;
      S[2 * k + 1] *= keep;
    };
    split_s(0);
    // the vector work on M and on the state's pieces runs beside the products of C and the state
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k + 1 < NK) load_c(k + 1);
      fetch(next, k, NK);
      stage();
      if (k + 1 < NK) split_s(k + 1);
      if (k < MW) put_m(k);
      mma_rows<QT>(Y, Sf[k & 1], cf[k & 1]);
      interleave<QT * 3 * (NP == 1 ? 1 : 2), NP == 1 ? 10 : 5>();
      stage();
    }
#pragma unroll
    for (int e = NK; e < MW; ++e) put_m(e);
    __syncthreads();
    const bool bad = bad_[c & 1] != 0;
    advance();
#pragma unroll
    for (int it = 0; it < QT; ++it) Y[it] *= since_[16 * it + lr];
    if (!bad) {
      load_x();
#pragma unroll
      for (int k = 0; k < Q / 32; ++k) {
        weigh_x(k);
#pragma unroll
        for (int it = 2 * k; it < QT; it += 2) {  // two token tiles at a time, from the block of 32 columns on
          Frag<3> mf[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) mf[r] = along<3>(Ms + 16 * (it + r) * LM + 32 * k, LM, nM, lane);
          mma_rows<2>(Y + it, xf[k], mf);
        }
      }
    } else {  // an infinity or a NaN times the zeros of M would reach earlier tokens: only j <= i
      load_x();
#pragma unroll
      for (int k = 0; k < Q / 32; ++k) weigh_x(k);
#pragma unroll
      for (int it = 0; it < QT; ++it)
        for (int j = 0; j <= 16 * it + lr; ++j) {
          const uint16_t* mp = Ms + (16 * it + lr) * LM + across_order(j);
          const float m = bf16_to_f32(mp[0]) + bf16_to_f32(mp[nM]) + bf16_to_f32(mp[2 * nM]);
          for (int k = NP - 1; k >= 0; --k) {
            const uint2 q = *(const uint2*)(Xs + k * nX + j * LX + 16 * wave + 4 * lg);
            Y[it][0] = fmaf(m, bf16lo(q.x), Y[it][0]);
            Y[it][1] = fmaf(m, bf16hi(q.x), Y[it][1]);
            Y[it][2] = fmaf(m, bf16lo(q.y), Y[it][2]);
            Y[it][3] = fmaf(m, bf16hi(q.y), Y[it][3]);
          }
        }
    }
    const rsrc_t to = block_rows(orow, (uint32_t)(rows * P) * 4);
#pragma unroll
    for (int it = 0; it < QT; ++it)
      store16(to, ooff + (uint32_t)(16 * it * P) * 4, 16 * it + lr < here ? Y[it] : f32x4_t{0.f, 0.f, 0.f, 0.f});
    // the state at the block's end
    constexpr int MH = NT < 4 ? NT : 4;  // tiles of d_k at a time
    Frag<NP> bf[MH];
    auto load_b = [&](int s) {  // step s: 32 tokens, MH tiles
      const int k = s / (NT / MH), m0 = s % (NT / MH) * MH;
#pragma unroll
      for (int m = 0; m < MH; ++m)
        bf[m] = across<NP, 8>(Bs + 32 * k * LB + 32 * ((m0 + m) >> 1) + 4 * (m & 1), LB, nB, lane);
    };
#pragma unroll
    for (int s = 0; s < Q / 32 * (NT / MH); ++s) {
      load_b(s);
      mma_cols<MH>(S + s % (NT / MH) * MH, bf, xw[s / (NT / MH)]);
    }
  }
  float* to = seg + 1 == L.segments ? A.s_out : nullptr;
  if (to && p < P) {
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int k = state_at(m);
      if (k < N) *(f32x4_t*)(to + srow + k) = S[m];
    }
  }
}

// ------------------------------------------------------------------ single tokens
// The state goes through the registers once, 16 bytes a lane; LR lanes hold a channel's row. Memory bounds it:
// 64 sequences, 16 heads of 128 x 128 (135 MB) take 31 us, 4.3 TB/s.
template <bool BF16, int LR>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs A) {
  constexpr int RW = 64 / LR;  // rows per wave
  const int blocks = (A.P + 4 * RW - 1) / (4 * RW);
  const int bh = blockIdx.x / blocks, b = bh / A.H, h = bh % A.H, g = h / (A.H / A.G);
  const int lane = threadIdx.x & 63, k = (lane % LR) * 4;
  const int p = (int)(blockIdx.x % blocks) * 4 * RW + (int)(threadIdx.x >> 6) * RW + lane / LR;
  const bool live = p < A.P && k < A.N;
  float* row = A.s_out + ((long long)bh * A.P + p) * A.N + k;
  f32x4_t s = live ? *(const f32x4_t*)row : f32x4_t{0.f, 0.f, 0.f, 0.f};
  const float dtv = softplus(A.dt[b * A.ld_dt + h] + A.dt_bias[h]);
  const float a = expf(fmaxf(-expf(A.A_log[h]) * dtv, -kMaxDecay));
  float o = 0.f, x = 0.f;
  if (live) {
    x = scan_val<BF16>(A.x, b * A.ld_x + h * A.P + p);
    const float w = dtv * x;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s[u] = fmaf(a, s[u], w * scan_val<BF16>(A.Bm, b * A.ld_b + g * A.N + k + u));
      o = fmaf(s[u], scan_val<BF16>(A.Cm, b * A.ld_c + g * A.N + k + u), o);
    }
    *(f32x4_t*)row = s;
  }
#pragma unroll
  for (int m = 1; m < LR; m <<= 1) o = add_xor_f32(o, m);
  if (live && k == 0) A.o[(long long)bh * A.P + p] = fmaf(A.D ? A.D[h] : 0.f, x, o);
}

// What a call split into s segments takes, in us at d_k 128: a block of this kernel takes 4 where a workgroup has
// its compute unit for itself and 6.5 where two share it, a block of the walk 2.4; walk and join start in 9 and
// move four states per segment. So 8 x 4096 tokens of 16 heads (128 units of 64 channels) run in 4 segments (145
// us; 246 in one), but 16 x 2000 tokens in one (133; 143 in two), and 16 x 100 too (20; 41 in two).
double split_cost(const sdm_scan_shape& S, long long units, int blocks, int s) {
  const int run = (blocks + s - 1) / s;
  const double block = units * s <= 256 ? 4.0 : 6.5 * (double)((units * s + 511) / 512);
  if (s == 1) return run * block;
  return run * (block + 2.4) + 9.0 + s / 8.0 + (double)s * S.B * S.H * S.d_v * S.d_k * 16.0 / 4.5e6;
}

ScanPlan plan_of(const sdm_scan_shape& S) {
  const int Q = S.in_dtype == SDM_BF16 ? block_tokens<true>() : block_tokens<false>();
  ScanPlan L;
  L.pblocks = (S.d_v + kPB - 1) / kPB;
  L.blocks = (S.T + Q - 1) / Q;
  const long long units = (long long)S.B * S.H * L.pblocks;
  L.segments = 1;
  for (int s = scan_segments(units, L.blocks, 512); s > 1; s /= 2)  // up to two workgroups per compute unit
    if (split_cost(S, units, L.blocks, s) < split_cost(S, units, L.blocks, L.segments)) L.segments = s;
  return L;
}

size_t workspace(const sdm_scan_shape& S, const ScanPlan& L, char* base, ScanGates* R, ScanWs* W) {
  const size_t units = (size_t)S.B * S.H, gb = gates_bytes(units, S.T, base, R);
  if (L.segments < 2) return gb;
  const size_t st = align_up(units * L.segments * S.d_v * S.d_k * 4);
  W->first = (float*)(base + gb);
  W->decay = (double*)(base + gb + st);
  return gb + st + align_up(units * L.segments * 8);
}

template <bool BF16, int NK>
hipError_t launch_blocks(const ScanArgs& A, const ScanPlan& L, const ScanGates& R, const ScanWs& W,
                         hipStream_t stream) {
  hipError_t e = launch_scan_gates(A, block_tokens<BF16>(), R, stream);
  if (e != hipSuccess) return e;
  if (L.segments > 1) {
    ScanWalk K{};
    K.B = A.B;
    K.T = A.T;
    K.H = A.H;
    K.G = A.G;
    K.N = A.N;
    K.P = A.P;
    K.blocks = L.blocks;
    K.segments = L.segments;
    K.stride = R.stride;
    K.X = A.x;
    K.K = A.Bm;
    K.xb = (long long)A.T * A.ld_x;
    K.xh = A.P;
    K.ld_x = A.ld_x;
    K.ld_k = A.ld_b;
    K.lengths = A.lengths;
    K.weight = R.left;
    K.l = R.l;
    K.start = A.s_in;
    K.first = W.first;
    K.decay = W.decay;
    e = launch_scan_walk(K, BF16, stream);
    if (e != hipSuccess) return e;
  }
  constexpr int lds = Tiles<BF16, NK>::bytes;
  const long long units = (long long)A.B * A.H * L.pblocks;
  hipLaunchKernelGGL((scan_kernel<BF16, NK>), dim3((unsigned)(units * L.segments)), dim3(256), lds, stream, A, L, W, R);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_step(const ScanArgs& A, hipStream_t stream) {
  const int quads = A.N / 4;
#define SDM_STEP(LR)                                                                                      \
  if (quads <= LR) {                                                                                      \
    const int rows = 4 * (64 / LR);                                                                       \
    const long long blocks = (long long)A.B * A.H * ((A.P + rows - 1) / rows);                            \
    hipLaunchKernelGGL((scan_step_kernel<BF16, LR>), dim3((unsigned)blocks), dim3(256), 0, stream, A); \
    return hipGetLastError();                                                                             \
  }
  SDM_STEP(2) SDM_STEP(4) SDM_STEP(8) SDM_STEP(16) SDM_STEP(32)
#undef SDM_STEP
  return hipErrorInvalidValue;
}

}  // namespace

size_t scan_workspace_bytes(const sdm_scan_shape& S) {
  ScanGates R;
  ScanWs W;
  return workspace(S, plan_of(S), nullptr, &R, &W);
}

hipError_t launch_scan(const sdm_scan_shape& S, const ScanArgs& A, hipStream_t stream) {
  const ScanPlan L = plan_of(S);
  ScanGates R;
  ScanWs W{};
  workspace(S, L, (char*)A.ws, &R, &W);
  const int steps = (A.N + 31) / 32;
  if (A.bf16)
    return steps == 1   ? launch_blocks<true, 1>(A, L, R, W, stream)
           : steps == 2 ? launch_blocks<true, 2>(A, L, R, W, stream)
                        : launch_blocks<true, 4>(A, L, R, W, stream);
  return steps == 1   ? launch_blocks<false, 1>(A, L, R, W, stream)
         : steps == 2 ? launch_blocks<false, 2>(A, L, R, W, stream)
                      : launch_blocks<false, 4>(A, L, R, W, stream);
}

hipError_t launch_scan_step(const ScanArgs& A, hipStream_t stream) {
  return A.bf16 ? launch_step<true>(A, stream) : launch_step<false>(A, stream);
}

}  // namespace sdm
