// Device helpers shared by the SDM kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {

constexpr int kWave = 64;

// ------------------------------------------------------------------ bf16 / float32 values
__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// Two float32 values -> two bfloat16 in one word (lo in bits 15:0), rounded to nearest even
// by gfx950's packed conversion instruction (v_cvt_pk_bf16_f32).
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// ------------------------------------------------------------------ wave primitives
__device__ __forceinline__ int lane_id() { return __lane_id(); }

// Exchange with lane ^ mask, for mask a power of two up to 32, without going through LDS
// addressing: DPP for masks 1, 2, 4 (half-row mirror then quad reversal), 8 (row rotate),
// ds_swizzle for 16, v_permlane32_swap for 32. `mask` must fold to a constant.
__device__ __forceinline__ uint32_t shfl_xor_u32(uint32_t v, int mask) {
  switch (mask) {
    case 1: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);  // quad_perm [1,0,3,2]
    case 2: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);  // quad_perm [2,3,0,1]
    case 4: return (uint32_t)__builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false), 0x1B,
                                                      0xF, 0xF, false);                // half mirror, quad reverse
    case 8: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false);  // row_ror:8
    case 16: return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F);              // swap 16
    case 32: {
      auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      return __lane_id() < 32 ? r[1] : r[0];
    }
    default: return (uint32_t)__shfl_xor((int)v, mask, kWave);
  }
}
__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int mask) {
  uint32_t lo = shfl_xor_u32((uint32_t)v, mask);
  uint32_t hi = shfl_xor_u32((uint32_t)(v >> 32), mask);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float shfl_xor_f32(float v, int mask) {
  return __uint_as_float(shfl_xor_u32(__float_as_uint(v), mask));
}

// v + (v of lane ^ mask), for mask a power of two up to 32 (fold to a constant). Within a
// row of 16 lanes the partner's value reaches the add through its DPP operand (one fused
// v_add_f32_dpp; every partner lies inside the row, so the zero that bound_ctrl gives an
// invalid source never occurs); mask 4 takes a half-row mirror first. The sum equals
// v + shfl_xor_f32(v, mask) bit for bit.
__device__ __forceinline__ float add_xor_f32(float v, int mask) {
  const int x = __float_as_int(v);
  switch (mask) {
    case 1: return v + __int_as_float(__builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true));  // quad_perm [1,0,3,2]
    case 2: return v + __int_as_float(__builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true));  // quad_perm [2,3,0,1]
    case 4: {
      const int t = __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false);                            // half mirror
      return v + __int_as_float(__builtin_amdgcn_update_dpp(0, t, 0x1B, 0xF, 0xF, true));         // quad reverse
    }
    case 8: return v + __int_as_float(__builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, true));  // row_ror:8
    default: return v + shfl_xor_f32(v, mask);
  }
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = add_xor_f32(v, m);
  return v;
}

__device__ __forceinline__ uint64_t ballot(bool p) { return __ballot(p); }
__device__ __forceinline__ int popc64(uint64_t m) { return __popcll(m); }
// number of set bits of m in lanes below this lane
__device__ __forceinline__ int mbcnt(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// 1 / (1 + exp(-x)) on the hardware's exp2 and reciprocal (about 1 step each; the argument's rounding adds
// |x| half steps to a value that is then below exp(-|x|))
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// ------------------------------------------------------------------ rows of 8 values
// 8 consecutive values of a bf16 or float32 row (16-byte aligned) as float32, and back.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, long long at, float (&v)[8]) {
  if (BF16) {
    const uint4 q = *(const uint4*)((const uint16_t*)base + at);
    v[0] = bf16lo(q.x); v[1] = bf16hi(q.x); v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
    v[4] = bf16lo(q.z); v[5] = bf16hi(q.z); v[6] = bf16lo(q.w); v[7] = bf16hi(q.w);
  } else {
    const float4 a = *(const float4*)((const float*)base + at), b = *(const float4*)((const float*)base + at + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* base, long long at, const float (&v)[8]) {
  if (BF16) {
    *(uint4*)((uint16_t*)base + at) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    *(float4*)((float*)base + at) = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)((float*)base + at + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Tokens of sequence b: its length clamped to [0, T], T where no lengths are given.
__device__ __forceinline__ int sequence_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// The rows of a block as a buffer: 16 bytes from an offset, zeros from `bytes` on, where stores are dropped.
// Rows behind a sequence's end and columns that are not there (kNowhere) so need no branch and no 64-bit
// address of their own; and a wave waits for its older loads alone, where a branch around newer accesses would
// have it wait for those too.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ rsrc_t block_rows(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint4 load16(rsrc_t rows, uint32_t at) {
  const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)at, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void store16(rsrc_t rows, uint32_t at, f32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rows, (int)at, 0, 0);
}

}  // namespace sdm
