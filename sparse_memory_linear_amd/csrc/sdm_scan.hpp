// What the forward and the backward pass of the selective scan share.
#pragma once

#include "sdm_device.hpp"
#include "sdm_internal.hpp"

namespace sdm {

constexpr int kScanBlock = 64;        // tokens per block: one per lane of a wave
constexpr float kMaxDecay = 1000.f;  // floor of a token's log-decay (exp(-1000) is 0 in float32)

template <bool BF16>
__device__ __forceinline__ float scan_val(const void* p, long long at) {
  return BF16 ? bf16_to_f32(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}

__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

}  // namespace sdm
