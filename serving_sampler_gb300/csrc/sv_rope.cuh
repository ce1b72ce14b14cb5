// What the rotary cache writes share: the angle of a pair, the place of a slot, packed
// 16-bit entries, and which vectors of a head make an item.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int kRopeThreads = 128;
constexpr int kRopeTokens = 4;  // most tokens of a CTA

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

struct RopeGeom {
    int32_t vecs;               // 16-byte vectors of a head
    int32_t half;               // rotated pairs
    int32_t rows;               // q heads, then k heads, then v heads
    int32_t items, line;        // items of a head, of a token
    uint32_t by_items;          // ceil(2^32 / items), for division by multiplication (0 for one item)
    int32_t tokens;             // of a CTA
    float by_dim;               // 1 / head_dim
};

// Items of a head: their two vectors, and the first of the eight pairs they hold (-1: they pass).
struct RopeItem {
    int32_t token, row, a, b, pair;
};
template <bool SIDE>
__device__ __forceinline__ RopeItem item_of(const RopeArgs& a, const RopeGeom& g, uint32_t x)
{
    RopeItem m;
    uint32_t in = x;
    m.token = 0;
#pragma unroll
    for (int i = 1; i < kRopeTokens; ++i) {
        if (in >= static_cast<uint32_t>(g.line)) {
            in -= g.line;
            ++m.token;
        }
    }
    m.row = static_cast<int32_t>(g.by_items != 0 ? __umulhi(in, g.by_items) : in);
    const int32_t j = static_cast<int32_t>(in - m.row * g.items);
    const bool turns = m.row < a.q.heads + a.cache.kv_heads;
    const int32_t cut = g.half / 8;  // rotated items when the halves lie apart
    m.a = 2 * j;
    m.b = 2 * j + 1;
    m.pair = -1;
    if (turns && SIDE) {
        m.pair = 8 * j;
    } else if (turns && j < cut) {
        m.a = j;
        m.b = j + cut;
        m.pair = 8 * j;
    }
    return m;
}

}  // namespace sv
