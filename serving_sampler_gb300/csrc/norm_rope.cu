// sv_norm_rope_cache: an RMS norm of every q and k head, rotary positions, k and v
// written into the paged cache, one read and one write of every head.
//
// y = x * (mean(x^2) + eps)^(-1/2) * w, then pairs of y turn as in rope.cu.  The sum of
// squares needs a whole head before its first entry can be written, so a head belongs to
// the 1, 2, 4 or 8 lanes that hold its vectors two by two (the same two of every head:
// the halves of eight pairs, or neighbours), and the sum is taken by exchanges among them.
#include <algorithm>

#include "sv_internal.h"
#include "sv_rope.cuh"

namespace sv {
namespace {

__device__ __forceinline__ float weight_at(const void* w, int32_t dtype, int i)
{
    if (w == nullptr) return 1.0f;
    if (dtype == SV_F32) return static_cast<const float*>(w)[i];
    if (dtype == SV_F16) return __half2float(static_cast<const __half*>(w)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// SIDE: as in rope.cu.  LANES: lanes of a head.
template <bool F16, bool SIDE, int LANES>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs n, const RopeGeom g)
{
    constexpr int kGroups = kRopeThreads / LANES;
    const RopeArgs& a = n.rope;
    __shared__ __align__(16) float2 s_cs[kRopeTokens][SV_MAX_HEAD_DIM / 2 + 8];
    __shared__ __align__(16) float s_w[2][SV_MAX_HEAD_DIM];
    __shared__ int64_t s_at[kRopeTokens];
    const int tid = threadIdx.x, j = tid % LANES;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * g.tokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(g.tokens), a.q.tokens - t0));
    const int Hq = a.q.heads, Hk = a.cache.kv_heads, D = a.cache.head_dim;
    const uint32_t total = static_cast<uint32_t>(tokens) * g.rows, step = kGroups * gridDim.y;

    // the two vectors of this lane, and the first of the eight pairs in them
    const int cut = g.half / 8;
    int va_at = 2 * j, vb_at = 2 * j + 1, pair = -1;
    if (SIDE) {
        pair = 8 * j < g.half ? 8 * j : -1;
    } else if (j < cut) {
        va_at = j;
        vb_at = j + cut;
        pair = 8 * j;
    }
    const bool has_a = va_at < g.vecs, has_b = vb_at < g.vecs;

    auto place = [&](uint32_t x, int& token, int& row) {
        uint32_t in = x;
        token = 0;
#pragma unroll
        for (int i = 1; i < kRopeTokens; ++i) {
            if (in >= static_cast<uint32_t>(g.rows)) {
                in -= g.rows;
                ++token;
            }
        }
        row = static_cast<int>(in);
    };
    auto load = [&](uint32_t x, uint4& va, uint4& vb) {
        va = vb = make_uint4(0, 0, 0, 0);
        if (x >= total) return;
        int token, row;
        place(x, token, row);
        const sv_heads& h = row < Hq ? a.q : row < Hq + Hk ? a.k : a.v;
        const int r = row < Hq ? row : row < Hq + Hk ? row - Hq : row - Hq - Hk;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(h.data) +
                                                          (t0 + token) * h.token_stride + r * h.head_stride);
        if (has_a) va = src[va_at];
        if (has_b) vb = src[vb_at];
    };
    uint4 na, nb;  // the next head's vectors, in flight
    uint32_t x = blockIdx.y * kGroups + tid / LANES;
    load(x, na, nb);
    if (tid < tokens) s_at[tid] = slot_offset(a, a.slot[t0 + tid]);
    for (int i = tid; i < D; i += kRopeThreads) {
        s_w[0][i] = weight_at(n.q_weight, n.weight_dtype, i);
        s_w[1][i] = weight_at(n.k_weight, n.weight_dtype, i);
    }
    for (int y = tid; y < tokens * g.half; y += kRopeThreads) {
        const int i = y / g.half, p = y - i * g.half;
        s_cs[i][p] = turn_of(a, a.position[t0 + i], p);
    }
    __syncthreads();

    // every thread of the CTA takes the same number of rounds: the exchanges need whole warps
    const uint32_t first = blockIdx.y * kGroups;
    for (uint32_t base = first; base < total; base += step, x += step) {
        const uint4 va = na, vb = nb;
        load(x + step, na, nb);
        float f[16];
        const uint32_t w[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 v = unpack2<F16>(w[e]);
            f[2 * e] = v.x;
            f[2 * e + 1] = v.y;
            sum = fmaf(v.x, v.x, sum);
            sum = fmaf(v.y, v.y, sum);
        }
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        int token, row;
        place(x, token, row);
        uint4 oa = va, ob = vb;
        if (x < total && row < Hq + Hk) {
            const float r = rsqrtf(sum * g.by_dim + n.eps);
            const float* weight = s_w[row < Hq ? 0 : 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (has_a) {
                    const float2 u = *reinterpret_cast<const float2*>(weight + 8 * va_at + 2 * e);
                    f[2 * e] *= r * u.x;
                    f[2 * e + 1] *= r * u.y;
                }
                if (has_b) {
                    const float2 u = *reinterpret_cast<const float2*>(weight + 8 * vb_at + 2 * e);
                    f[8 + 2 * e] *= r * u.x;
                    f[8 + 2 * e + 1] *= r * u.y;
                }
            }
            if (pair >= 0) {
                const float4* cs = reinterpret_cast<const float4*>(&s_cs[token][pair]);
                if (SIDE) {
                    // the last rotated vectors may hold fewer than eight pairs: the others pass
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 f2 = cs[e / 2];
                        const float c = e & 1 ? f2.z : f2.x, s = e & 1 ? f2.w : f2.y;
                        const float u = f[2 * e], v = f[2 * e + 1];
                        if (pair + e < g.half) {
                            f[2 * e] = fmaf(-v, s, u * c);
                            f[2 * e + 1] = fmaf(u, s, v * c);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 f2 = cs[e / 2];
                        const float c = e & 1 ? f2.z : f2.x, s = e & 1 ? f2.w : f2.y;
                        const float u = f[e], v = f[8 + e];
                        f[e] = fmaf(-v, s, u * c);
                        f[8 + e] = fmaf(u, s, v * c);
                    }
                }
            }
            oa = make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]),
                            pack2<F16>(f[6], f[7]));
            ob = make_uint4(pack2<F16>(f[8], f[9]), pack2<F16>(f[10], f[11]), pack2<F16>(f[12], f[13]),
                            pack2<F16>(f[14], f[15]));
        }
        if (x >= total) continue;
        uint4* dst;
        if (row < Hq) {
            dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) +
                                           (t0 + token) * a.q_out.token_stride + row * a.q_out.head_stride);
        } else {
            const int64_t at = s_at[token];
            if (at < 0) continue;
            const bool key = row < Hq + Hk;
            dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(key ? a.cache.k : a.cache.v) + at +
                                           (row - (key ? Hq : Hq + Hk)) * a.cache.head_stride);
        }
        if (has_a) dst[va_at] = oa;
        if (has_b) dst[vb_at] = ob;
    }
}

// Halves that lie apart by no multiple of 8 entries: a warp takes a head, entry by entry, and
// gets the partners' values by a second read of them; it has read all before it writes any.
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_entries_kernel(const __grid_constant__ NormRopeArgs n,
                                                                         const RopeGeom g)
{
    constexpr int kMost = SV_MAX_HEAD_DIM / 32;
    const RopeArgs& a = n.rope;
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int Hq = a.q.heads, Hk = a.cache.kv_heads, D = a.cache.head_dim;
    const int64_t at = slot_offset(a, a.slot[t]);
    auto widen = [](uint16_t w) { return unpack2<F16>(w).x; };
    float2 cs[kMost];
#pragma unroll
    for (int e = 0; e < kMost; ++e) {
        const int d = lane + 32 * e;
        if (d < 2 * g.half) cs[e] = turn_of(a, a.position[t], d < g.half ? d : d - g.half);
    }
    for (int row = threadIdx.x / 32 + blockIdx.y * (kRopeThreads / 32); row < g.rows;
         row += gridDim.y * (kRopeThreads / 32)) {
        const sv_heads& h = row < Hq ? a.q : row < Hq + Hk ? a.k : a.v;
        const int r = row < Hq ? row : row < Hq + Hk ? row - Hq : row - Hq - Hk;
        const uint16_t* src = static_cast<const uint16_t*>(h.data) + t * h.token_stride + r * h.head_stride;
        const bool normed = row < Hq + Hk;
        const void* weight = row < Hq ? n.q_weight : n.k_weight;
        uint16_t in[kMost];
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < kMost; ++e) {
            const int d = lane + 32 * e;
            in[e] = d < D ? src[d] : 0;
            const float v = widen(in[e]);
            sum = fmaf(v, v, sum);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (normed) {
            const float scale = rsqrtf(sum * g.by_dim + n.eps);
#pragma unroll
            for (int e = 0; e < kMost; ++e) {
                const int d = lane + 32 * e;
                if (d >= D) continue;
                float v = widen(in[e]) * (scale * weight_at(weight, n.weight_dtype, d));
                if (d < 2 * g.half) {
                    const bool low = d < g.half;
                    const int o = low ? d + g.half : d - g.half;
                    const float y = widen(src[o]) * (scale * weight_at(weight, n.weight_dtype, o));
                    v = fmaf(low ? -y : y, cs[e].y, v * cs[e].x);
                }
                in[e] = static_cast<uint16_t>(pack2<F16>(v, 0.0f));
            }
        }
        __syncwarp();
        uint16_t* dst = row < Hq ? static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) + t * a.q_out.token_stride +
                                       r * a.q_out.head_stride
                                 : static_cast<uint16_t*>(normed ? a.cache.k : a.cache.v) + at + r * a.cache.head_stride;
        if (row < Hq || at >= 0) {
#pragma unroll
            for (int e = 0; e < kMost; ++e)
                if (lane + 32 * e < D) dst[lane + 32 * e] = in[e];
        }
    }
}

template <bool F16, bool SIDE>
void launch_lanes(const NormRopeArgs& n, const RopeGeom& g, int lanes, dim3 grid, cudaStream_t stream)
{
    if (lanes == 1)
        norm_rope_kernel<F16, SIDE, 1><<<grid, kRopeThreads, 0, stream>>>(n, g);
    else if (lanes == 2)
        norm_rope_kernel<F16, SIDE, 2><<<grid, kRopeThreads, 0, stream>>>(n, g);
    else if (lanes == 4)
        norm_rope_kernel<F16, SIDE, 4><<<grid, kRopeThreads, 0, stream>>>(n, g);
    else
        norm_rope_kernel<F16, SIDE, 8><<<grid, kRopeThreads, 0, stream>>>(n, g);
}

}  // namespace

cudaError_t launch_norm_rope_cache(const NormRopeArgs& n, cudaStream_t stream)
{
    const RopeArgs& a = n.rope;
    RopeGeom g{};
    g.vecs = a.cache.head_dim / 8;
    g.half = a.rot_dim / 2;
    g.rows = a.q.heads + 2 * a.cache.kv_heads;
    g.by_dim = 1.0f / a.cache.head_dim;
    const int sms = device_sm_count();
    const bool f16 = a.cache.dtype == SV_F16;
    auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    if (!a.interleaved && g.half % 8 != 0) {
        const int64_t most = cdiv(g.rows, kRopeThreads / 32), want = cdiv(8 * sms, a.q.tokens);
        const dim3 grid(static_cast<unsigned>(a.q.tokens), static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
        if (f16)
            norm_rope_entries_kernel<true><<<grid, kRopeThreads, 0, stream>>>(n, g);
        else
            norm_rope_entries_kernel<false><<<grid, kRopeThreads, 0, stream>>>(n, g);
        return cudaGetLastError();
    }
    int lanes = 1;
    while (2 * lanes < g.vecs) lanes *= 2;
    g.tokens = a.q.tokens >= kRopeTokens * 8 * sms ? kRopeTokens : 1;
    const int64_t most = cdiv(static_cast<int64_t>(g.tokens) * g.rows, kRopeThreads / lanes);
    const int64_t want = cdiv(2 * sms, a.q.tokens);
    const dim3 grid(static_cast<unsigned>(cdiv(a.q.tokens, g.tokens)),
                    static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
    if (a.interleaved) {
        if (f16)
            launch_lanes<true, true>(n, g, lanes, grid, stream);
        else
            launch_lanes<false, true>(n, g, lanes, grid, stream);
    } else {
        if (f16)
            launch_lanes<true, false>(n, g, lanes, grid, stream);
        else
            launch_lanes<false, false>(n, g, lanes, grid, stream);
    }
    return cudaGetLastError();
}

}  // namespace sv
