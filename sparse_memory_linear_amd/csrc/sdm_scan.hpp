// What the forward and the backward pass of the selective scan share: the factors of the matrix
// products as bf16 pieces, the reads of operand fragments, the log-decays of a block of tokens.
//
// v_mfma_f32_16x16x32_bf16: D[row][col] += sum over k of A[row][k] B[k][col]. Lane l gives A's row (B's
// column) l % 16 for 8 of the 32 k; the same choice of k for A and B pairs them up whatever the
// instruction's own order is. Of D the lane holds column l % 16, rows 4 (l / 16) + 0..3.
//
// A float32 factor enters as three bf16 pieces that add up to it exactly (each takes the next 8 of the 24
// bits), a bf16 factor as itself. The product of two factors of n_a and n_b pieces is the sum of the
// products of the pieces whose ranks add up to at most 2; what is left out is below 2^-23 of it.
#pragma once

#include "sdm_device.hpp"
#include "sdm_internal.hpp"

namespace sdm {

constexpr float kMaxDecay = 1000.f;  // floor of a token's log-decay (exp(-1000) is 0 in float32)
constexpr double kLog2e = 1.4426950408889634074;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ float scan_val(const void* p, long long at) {
  return BF16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}

__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f((float)x); }

// High halves of two words as one word (a in the low half)
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float truncated(float a) { return __uint_as_float(__float_as_uint(a) & 0xFFFF0000u); }

// Two float32 values as three words of two bf16 pieces each
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[3]) {
  w[0] = high_halves(a, b);
  a -= truncated(a);
  b -= truncated(b);
  w[1] = high_halves(a, b);
  a -= truncated(a);
  b -= truncated(b);
  w[2] = high_halves(a, b);
}

// One operand fragment: 8 bf16 of each of NP pieces
template <int NP>
struct Frag {
  uint4 v[NP];
};

// 8 float32 values as a fragment of three pieces
__device__ __forceinline__ Frag<3> split8(const float (&x)[8]) {
  Frag<3> f;
  uint32_t w[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_pair(x[2 * i], x[2 * i + 1], w[i]);
#pragma unroll
  for (int k = 0; k < 3; ++k) f.v[k] = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
  return f;
}

// The 8 values of a fragment (the sum of its pieces)
template <int NP>
__device__ __forceinline__ void values_of(const Frag<NP>& f, float (&x)[8]) {
#pragma unroll
  for (int k = NP - 1; k >= 0; --k) {
    const uint32_t w[4] = {f.v[k].x, f.v[k].y, f.v[k].z, f.v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = bf16lo(w[i]), hi = bf16hi(w[i]);
      x[2 * i] = k == NP - 1 ? lo : x[2 * i] + lo;
      x[2 * i + 1] = k == NP - 1 ? hi : x[2 * i + 1] + hi;
    }
  }
}

template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4_t& d, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j <= 2)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v[i]),
                                                    __builtin_bit_cast(bf16x8_t, b.v[j]), d, 0, 0, 0);
}

// The same for N results at once with one common operand each way: neighbouring instructions add to
// different results, so none waits for the one before. d[i] += a_i b_i with a or b the same for all.
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_rows(f32x4_t* d, const Frag<NA>& a, const Frag<NB>* b) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (i + j <= 2)
          d[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v[i]),
                                                         __builtin_bit_cast(bf16x8_t, b[r].v[j]), d[r], 0, 0, 0);
}
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_cols(f32x4_t* d, const Frag<NA>* a, const Frag<NB>& b) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
#pragma unroll
      for (int r = 0; r < N; ++r)
        if (i + j <= 2)
          d[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[r].v[i]),
                                                         __builtin_bit_cast(bf16x8_t, b.v[j]), d[r], 0, 0, 0);
}

// Keeps reads that are written ahead of the products of the step before ahead of them
__device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }

// Asks for an order of `M` matrix instructions with V vector instructions behind each: a wave issues in
// order, so only what is written between them runs beside them
template <int M, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
  }
}

// Reads of fragments from a tile in LDS, rows `ld` bf16 apart, planes (pieces) `plane` apart.
//
// along(): row l % 16 of the tile is the operand's row, k runs along it: lanes with g = l / 16 take the
// 8 k from 8 g.
template <int NP>
__device__ __forceinline__ Frag<NP> along(const uint16_t* tile, int ld, int plane, int lane) {
  Frag<NP> f;
  const uint16_t* p = tile + (lane & 15) * ld + (lane >> 4) * 8;
#pragma unroll
  for (int k = 0; k < NP; ++k) f.v[k] = *(const uint4*)(p + k * plane);
  return f;
}
// across(): a column of the tile is the operand's row, k runs over the tile's rows: lanes with g = l / 16
// take rows 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3. The transposing read hands 16 lanes the columns of
// four rows of four runs of 4 values, which the lanes address. RUN = 4: lane l has column l % 16.
// RUN = 8: column 8 ((l % 16) / 4) + l % 4, so that this tile and the one 4 columns on are the even and
// the odd 16 rows of a result whose lanes, with the two stacked, hold the 8 consecutive k of along().
template <int NP, int RUN = 4>
__device__ __forceinline__ Frag<NP> across(uint16_t* tile, int ld, int plane, int lane) {
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  Frag<NP> f;
  uint16_t* p = tile + ((lane >> 4) * 4 + ((lane >> 2) & 3)) * ld + (lane & 3) * RUN;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(p + k * plane)));
    const uint2 b =
        __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(p + k * plane + 16 * ld)));
    f.v[k] = make_uint4(a.x, a.y, b.x, b.y);
  }
  return f;
}
// Where column j of a block of 32 lies in a tile whose rows along() reads against rows that across()
// reads: the order of across() in runs of 4.
__device__ __forceinline__ int across_order(int j) {
  return (j & ~31) | ((j & 12) << 1) | ((j & 16) >> 2) | (j & 3);
}

// One step of a prefix sum: v plus the v that the DPP control hands this lane (0 where none, or where
// the row is not in ROWS)
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, true);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive sum over the lanes of a block up to this one: shifts by 1, 2, 4, 8 in the rows of 16 lanes,
// then the last lane of row 0 to row 1 and of row 2 to row 3, then lane 31 to rows 2 and 3
template <int Q>
__device__ __forceinline__ double block_prefix(double v) {  // of blocks of Q lanes, 32 or 64
  v = add_dpp<0x111, 0xF>(v);
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);
  return Q == 64 ? add_dpp<0x143, 0xC>(v) : v;
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// What the products take of the time steps, [B*H][blocks of 64 tokens * 64], padding as steps of 0:
// log2 of the decay summed over the token's block (of Q tokens), the step, and the decays as float32
// factors from the block's start to the token and from the token (times its step) to the block's end
struct ScanGates {
  double* l;
  float *step, *since, *left;
  int stride;  // tokens per row
};
inline size_t gates_bytes(long long units, int T, char* base, ScanGates* g) {
  const size_t stride = ((size_t)T + 63) / 64 * 64, n = (size_t)units * stride;
  g->stride = (int)stride;
  g->l = (double*)base;
  g->step = (float*)(base + n * 8);
  g->since = g->step + n;
  g->left = g->since + n;
  return align_up(n * 20);
}
hipError_t launch_scan_gates(const ScanArgs& A, int Q, const ScanGates& g, hipStream_t stream);

// Turned states, as the gradient's blocks take S: the operand pieces of its products in their lanes' order,
// [d_k / 16][d_v / 32][2 halves][64 lanes][4 channels], where lane 16 g + r has d_k r and channels 8 g .. 8 g + 7,
// with d_k up to 32, 64 or 128 and d_v up to a multiple of 64. A wave loads 1 KB in a row with each instruction;
// as [d_k][d_v] its lanes' pieces lay 512 bytes apart.
__host__ __device__ inline int turned_dk(int N) { return N <= 32 ? 32 : N <= 64 ? 64 : 128; }
__host__ __device__ inline int turned_dv(int P) { return (P + 63) / 64 * 64; }
__host__ __device__ inline int turned_size(int N, int P) { return turned_dk(N) * turned_dv(P); }
// (in floats; p in whole halves)
__device__ __forceinline__ int turned_at(int tile, int P, int p, int r) {
  return (((tile * (turned_dv(P) / 32) + p / 32) * 2 + p / 4 % 2) * 64 + p / 8 % 4 * 16 + r) * 4;
}

// One walk over the blocks (sdm_scan_states.hip): token t of (b, h) has X at b xb + h xh + t ld_x, K at
// (b T + t) ld_k + g N, its weight and log-decay at (b H + h) stride + t.
struct ScanWalk {
  int B, T, H, G, N, P, blocks, segments, segs, stride;
  const void *X, *K;
  long long xb, xh, ld_x, ld_k;
  const int32_t* lengths;
  const float* weight;
  const double* l;
  const float* start;  // state before the walk, or null
  float* end;          // state behind it, or null
  // of several segments: [segments + 1][B*H][P][N] states before them (forward with `states`: turned), the last
  // place for what the last one adds; and [segments + 1][B*H] log2 of the decay of the segment before
  float* first;
  double* decay;
  // [B*H][blocks] what the segment adds to the states entering the blocks, forward turned, backward [P][N], and
  // [B*H][blocks] the decay from the segment's start to there; null: only `first` is wanted
  float *states, *upto;
};
// Segments of a walk (or of the forward kernel): a call of few units is split until `wanted` workgroups are
// busy, but for s segments of n blocks the walk and the kernel behind it take about 4 us per block, n / s in a
// row, and the join 1 us per 8 segments, so s stays below sqrt(32 n): 25 us for 1024 tokens of 8 heads (36 with
// at least four blocks each), 99 us for 131072 tokens of one head (133 with 512 segments).
inline int scan_segments(long long units, int blocks, int wanted) {
  long long s = wanted / units;
  if (s > blocks) s = blocks;
  while (s * s > 32ll * blocks) --s;
  return s < 1 ? 1 : (int)s;
}
hipError_t launch_scan_walk(const ScanWalk& A, bool bf16, hipStream_t stream);
// The states of a forward walk A and, with the same sizes, of a walk back U, blocks of each
hipError_t launch_scan_walks(const ScanWalk& A, const ScanWalk& U, bool bf16, hipStream_t stream);

}  // namespace sdm
