// What the rotary cache writes share: the angle of a pair, the place of a slot and packed
// 16-bit entries.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int kRopeThreads = 128;

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// cosine and sine of pair `pair` at position p
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int32_t p, int pair)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(p)) * a.freqs[pair];
    const float turn = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(turn, &s, &c);
    return make_float2(c * a.mscale, s * a.mscale);
}

// The cache offset of a slot, -1 for one outside the cache.
__device__ __forceinline__ int64_t slot_offset(const RopeArgs& a, int64_t slot)
{
    const int64_t block = slot >= 0 ? slot / a.cache.block_size : -1;
    if (block < 0 || block >= a.cache.num_blocks) return -1;
    return block * a.cache.block_stride + (slot - block * a.cache.block_size) * a.cache.token_stride;
}

}  // namespace sv
