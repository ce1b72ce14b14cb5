// sv_rope_cache: rotary positions on q and k, k and v written into the paged
// cache, one read and one write of every head.
//
// The angle of pair i at position p is p * F_i turns, F_i a 64-bit fraction of a
// turn: the 64-bit product wraps at whole turns by itself, so its upper 32 bits
// are the angle to 2^-32 turns at any position, where an fp32 product of p and a
// frequency is off by p * 2^-24 radians.  They become a float in [-1, 1) half
// turns for sincospif.
//
// One CTA takes one token (and a share of its heads, when there are few tokens):
// rot_dim / 2 threads take the token's sines while everybody's first loads are in
// flight, then the CTA runs over (head, 16-byte vector).  A head is held by one
// group of lanes of a warp (head_dim / 8 rounded up to a power of two), and the
// other half of each pair comes from a lane of that group, so q may be rotated in
// place: a group has loaded its head before it stores any of it.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads a lane group has in flight

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
template <bool F16>
__device__ __forceinline__ float entry(const uint16_t* p)
{
    const uint32_t w = *p;
    return F16 ? unpack2<true>(w).x : __uint_as_float(w << 16);
}

struct RopeGeom {
    int32_t vecs;       // 16-byte vectors of a head
    int32_t group_log;  // log2 of the lanes that hold a head
    int32_t half;       // rotated pairs
    int32_t rows;       // q heads, then k heads, then v heads
    bool by_lanes;      // half layout whose partner vectors are whole: half % 8 == 0
};

template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) rope_cache_kernel(const RopeArgs a, const RopeGeom g)
{
    __shared__ float2 s_cs[SV_MAX_HEAD_DIM / 2];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int lane = tid & ((1 << g.group_log) - 1);
    const int groups = kRopeThreads >> g.group_log;
    const int stride = groups * gridDim.y;
    const bool on = lane < g.vecs;
    const int Hq = a.q.heads, Hk = a.cache.kv_heads;

    const int64_t slot = a.slot[t];
    const int64_t block = slot >= 0 ? slot / a.cache.block_size : -1;
    const bool cached = block >= 0 && block < a.cache.num_blocks;
    const int64_t cache_at = cached ? block * a.cache.block_stride +
                                          (slot - block * a.cache.block_size) * a.cache.token_stride
                                    : 0;

    auto source = [&](int row) -> const uint16_t* {
        if (row < Hq)
            return static_cast<const uint16_t*>(a.q.data) + t * a.q.token_stride + row * a.q.head_stride;
        if (row < Hq + Hk)
            return static_cast<const uint16_t*>(a.k.data) + t * a.k.token_stride + (row - Hq) * a.k.head_stride;
        return static_cast<const uint16_t*>(a.v.data) + t * a.v.token_stride + (row - Hq - Hk) * a.v.head_stride;
    };
    auto target = [&](int row) -> uint16_t* {
        if (row < Hq)
            return static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) + t * a.q_out.token_stride +
                   row * a.q_out.head_stride;
        if (!cached) return nullptr;
        if (row < Hq + Hk) return static_cast<uint16_t*>(a.cache.k) + cache_at + (row - Hq) * a.cache.head_stride;
        return static_cast<uint16_t*>(a.cache.v) + cache_at + (row - Hq - Hk) * a.cache.head_stride;
    };

    uint4 val[kRopeBatch];
    const int first = (tid >> g.group_log) + groups * blockIdx.y;
    auto load = [&](int row0) {
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            const int row = row0 + u * stride;
            val[u] = make_uint4(0, 0, 0, 0);
            if (on && row < g.rows) val[u] = *reinterpret_cast<const uint4*>(source(row) + lane * 8);
        }
    };
    load(first);
    if (tid < g.half) {
        const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(a.position[t])) * a.freqs[tid];
        const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
        float s, c;
        sincospif(x, &s, &c);
        s_cs[tid] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();

    const int shift = g.half / 8;  // vectors between the halves of a pair (by_lanes)
    const uint32_t all = 0xFFFFFFFFu;
    for (int row0 = first;; row0 += kRopeBatch * stride) {
        // every lane of a warp makes the same number of rounds: the group's first row decides
        if (__all_sync(all, row0 >= g.rows)) break;
        if (row0 != first) load(row0);
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            const int row = row0 + u * stride;
            const bool live = row < g.rows;
            uint32_t w[4] = {val[u].x, val[u].y, val[u].z, val[u].w};
            uint32_t o[4];
            if (g.by_lanes) {
                const bool low = lane < shift, rotated = lane < 2 * shift;
                const int other = (tid & 31 & ~((1 << g.group_log) - 1)) | (low ? lane + shift : rotated ? lane - shift : lane);
                uint32_t m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = __shfl_sync(all, w[i], other);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (rotated && live && row < Hq + Hk) {
                        const float2 x = unpack2<F16>(w[i]), y = unpack2<F16>(m[i]);
                        const int p = (low ? lane : lane - shift) * 8 + 2 * i;
                        const float2 e = s_cs[p], f = s_cs[p + 1];
                        const float se = low ? -e.y : e.y, sf = low ? -f.y : f.y;
                        o[i] = pack2<F16>(fmaf(y.x, se, x.x * e.x), fmaf(y.y, sf, x.y * f.x));
                    } else {
                        o[i] = w[i];
                    }
                }
            } else if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = lane * 4 + i;
                    if (p < g.half && live && row < Hq + Hk) {
                        const float2 x = unpack2<F16>(w[i]), e = s_cs[p];
                        o[i] = pack2<F16>(fmaf(-x.y, e.y, x.x * e.x), fmaf(x.x, e.y, x.y * e.x));
                    } else {
                        o[i] = w[i];
                    }
                }
            } else {
                // pairs that straddle vectors: partners read one by one (from L1, the group has the line)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (on && live && row < Hq + Hk) {
                        const uint16_t* src = source(row);
                        float y[2];
                        const float2 x = unpack2<F16>(w[i]);
                        const float v[2] = {x.x, x.y};
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int d = lane * 8 + 2 * i + q;
                            if (d < g.half) {
                                const float2 e = s_cs[d];
                                y[q] = fmaf(-entry<F16>(src + d + g.half), e.y, v[q] * e.x);
                            } else if (d < 2 * g.half) {
                                const float2 e = s_cs[d - g.half];
                                y[q] = fmaf(entry<F16>(src + d - g.half), e.y, v[q] * e.x);
                            } else {
                                y[q] = v[q];
                            }
                        }
                        o[i] = pack2<F16>(y[0], y[1]);
                    } else {
                        o[i] = w[i];
                    }
                }
                __syncwarp();  // partners are read before q is overwritten in place
            }
            if (on && live) {
                uint16_t* dst = target(row);
                if (dst != nullptr) *reinterpret_cast<uint4*>(dst + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_cache(const RopeArgs& a, cudaStream_t stream)
{
    RopeGeom g{};
    g.vecs = a.cache.head_dim / 8;
    while ((1 << g.group_log) < g.vecs) ++g.group_log;
    g.half = a.rot_dim / 2;
    g.rows = a.q.heads + 2 * a.cache.kv_heads;
    g.by_lanes = !a.interleaved && g.half % 8 == 0;
    // few tokens: their heads are spread over the SMs
    const int groups = kRopeThreads >> g.group_log;
    const int most = (g.rows + groups - 1) / groups;
    const int want = (device_sm_count() + a.q.tokens - 1) / a.q.tokens;
    const dim3 grid(static_cast<unsigned>(a.q.tokens), static_cast<unsigned>(std::max(1, std::min(want, most))));
    if (a.cache.dtype == SV_F16)
        rope_cache_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, g);
    else
        rope_cache_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
