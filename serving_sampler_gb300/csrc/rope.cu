// sv_rope_cache: rotary positions on q and k, k and v written into the paged
// cache, one read and one write of every head.
//
// The angle of pair i at position p is p * F_i turns, F_i a 64-bit fraction of a
// turn: the 64-bit product wraps at whole turns by itself, so its upper 32 bits
// are the angle to 2^-32 turns at any position, where an fp32 product of p and a
// frequency is off by p * 2^-24 radians.  They become a float in [-1, 1) half
// turns for sincospif.
//
// rope_cache_kernel: a CTA takes a few tokens.  Its threads take the sines of all of
// them while their first loads are in flight, then each takes items of two 16-byte
// vectors: the two halves of eight pairs (or eight pairs that lie side by side, or two
// vectors that pass), so that no entry has to come from another thread and q may be
// rotated in place.  Items of all heads of the CTA's tokens lie on one line, which
// keeps every lane busy for any head size.
//
// Bound by bytes where there are many: 47.7 us for the 284 MB of 60 x 257 tokens, 32 heads
// and 8 key heads of 96, 6.0 TB/s, 0.88 of a copy's rate; 14.9 us for the 77 MB of 64 x 65
// tokens, 28 heads and 4 key heads of 128, 5.1 TB/s; 2.6 us, a launch, for 9 tokens.  With
// one vector an item and the partners exchanged between lanes the first two took 96 and 23 us.
#include <algorithm>

#include "sv_internal.h"
#include "sv_rope.cuh"

namespace sv {
namespace {

constexpr int kRopeTokens = 4;  // most tokens of a CTA

struct RopeGeom {
    int32_t vecs;               // 16-byte vectors of a head
    int32_t half;               // rotated pairs
    int32_t rows;               // q heads, then k heads, then v heads
    int32_t items, line;        // items of a head, of a token
    uint32_t by_items;          // ceil(2^32 / items), for division by multiplication (0 for one item)
    int32_t tokens;             // of a CTA
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

// SIDE: the entries of a pair lie side by side; otherwise half a rotated part apart (a multiple of 8).
template <bool F16, bool SIDE>
__global__ void __launch_bounds__(kRopeThreads) rope_cache_kernel(const __grid_constant__ RopeArgs a, const RopeGeom g)
{
    __shared__ __align__(16) float2 s_cs[kRopeTokens][SV_MAX_HEAD_DIM / 2 + 8];
    __shared__ int64_t s_at[kRopeTokens];
    const int tid = threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * g.tokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(g.tokens), a.q.tokens - t0));
    const int Hq = a.q.heads, Hk = a.cache.kv_heads;
    const uint32_t total = static_cast<uint32_t>(tokens) * g.line, step = kRopeThreads * gridDim.y;

    auto load = [&](uint32_t x, uint4& va, uint4& vb) {
        if (x < total) {
            const RopeItem m = item_of<SIDE>(a, g, x);
            const sv_heads& h = m.row < Hq ? a.q : m.row < Hq + Hk ? a.k : a.v;
            const int row = m.row < Hq ? m.row : m.row < Hq + Hk ? m.row - Hq : m.row - Hq - Hk;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(h.data) +
                                                              (t0 + m.token) * h.token_stride + row * h.head_stride);
            va = src[m.a];
            if (m.b < g.vecs) vb = src[m.b];
        }
    };
    uint4 na, nb;  // the next item, in flight
    uint32_t x = blockIdx.y * kRopeThreads + tid;
    load(x, na, nb);
    if (tid < tokens) s_at[tid] = slot_offset(a, a.slot[t0 + tid]);
    for (int y = tid; y < tokens * g.half; y += kRopeThreads) {
        const int i = y / g.half, pair = y - i * g.half;
        s_cs[i][pair] = turn_of(a, a.position[t0 + i], pair);
    }
    __syncthreads();

    for (; x < total; x += step) {
        const uint4 va = na, vb = nb;
        load(x + step, na, nb);
        const RopeItem m = item_of<SIDE>(a, g, x);
        uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        if (m.pair >= 0) {
            const float4* cs = reinterpret_cast<const float4*>(&s_cs[m.token][m.pair]);
            if (SIDE) {
                // the last rotated item may hold fewer than eight pairs: the others pass
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint32_t& w = e < 4 ? wa[e] : wb[e - 4];
                    const float4 f2 = cs[e / 2];
                    const float c = e & 1 ? f2.z : f2.x, s = e & 1 ? f2.w : f2.y;
                    const float2 v = unpack2<F16>(w);
                    if (m.pair + e < g.half) w = pack2<F16>(fmaf(-v.y, s, v.x * c), fmaf(v.x, s, v.y * c));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 f = cs[e];  // two pairs
                    const float2 v = unpack2<F16>(wa[e]), w = unpack2<F16>(wb[e]);
                    wa[e] = pack2<F16>(fmaf(-w.x, f.y, v.x * f.x), fmaf(-w.y, f.w, v.y * f.z));
                    wb[e] = pack2<F16>(fmaf(v.x, f.y, w.x * f.x), fmaf(v.y, f.w, w.y * f.z));
                }
            }
        }
        uint4* dst;
        if (m.row < Hq) {
            dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) +
                                           (t0 + m.token) * a.q_out.token_stride + m.row * a.q_out.head_stride);
        } else {
            const int64_t at = s_at[m.token];
            if (at < 0) continue;
            const bool key = m.row < Hq + Hk;
            dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(key ? a.cache.k : a.cache.v) + at +
                                           (m.row - (key ? Hq : Hq + Hk)) * a.cache.head_stride);
        }
        dst[m.a] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
        if (m.b < g.vecs) dst[m.b] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
}

// Halves that lie apart by no multiple of 8 entries: a warp takes a head, entry by entry; it has
// read all of it before it writes any.  Bound by its 2-byte accesses, of which a rotated entry needs two:
// 36 us for the 58 MB of 64 x 65 tokens, 28 + 4 heads of 96 with 24 rotated, 1.6 TB/s, where
// rope_cache_kernel takes 14.8 with all 96 rotated; 31 us with 20 of 80.
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) rope_entries_kernel(const __grid_constant__ RopeArgs a, const RopeGeom g)
{
    constexpr int kMost = SV_MAX_HEAD_DIM / 32;
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
        uint16_t out[kMost];
#pragma unroll
        for (int e = 0; e < kMost; ++e) {
            const int d = lane + 32 * e;
            if (d < D) {
                out[e] = src[d];
                if (row < Hq + Hk && d < 2 * g.half) {
                    const bool low = d < g.half;
                    const float y = widen(src[low ? d + g.half : d - g.half]);
                    out[e] = static_cast<uint16_t>(pack2<F16>(fmaf(low ? -y : y, cs[e].y, widen(out[e]) * cs[e].x), 0.0f));
                }
            }
        }
        __syncwarp();
        uint16_t* dst = row < Hq ? static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) + t * a.q_out.token_stride +
                                       r * a.q_out.head_stride
                                 : static_cast<uint16_t*>(row < Hq + Hk ? a.cache.k : a.cache.v) + at + r * a.cache.head_stride;
        if (row < Hq || at >= 0) {
#pragma unroll
            for (int e = 0; e < kMost; ++e)
                if (lane + 32 * e < D) dst[lane + 32 * e] = out[e];
        }
    }
}

}  // namespace

cudaError_t launch_rope_cache(const RopeArgs& a, cudaStream_t stream)
{
    RopeGeom g{};
    g.vecs = a.cache.head_dim / 8;
    g.half = a.rot_dim / 2;
    g.rows = a.q.heads + 2 * a.cache.kv_heads;
    g.items = (g.vecs + 1) / 2;
    g.line = g.rows * g.items;
    // exact: at most 8 items, and fewer than 2^20 of a token (65,536 rows)
    g.by_items = g.items > 1 ? static_cast<uint32_t>((0x100000000ull + g.items - 1) / g.items) : 0u;
    const int sms = device_sm_count();
    const bool f16 = a.cache.dtype == SV_F16;
    auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    if (!a.interleaved && g.half % 8 != 0) {
        const int64_t most = cdiv(g.rows, kRopeThreads / 32), want = cdiv(8 * sms, a.q.tokens);
        const dim3 grid(static_cast<unsigned>(a.q.tokens), static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
        if (f16)
            rope_entries_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, g);
        else
            rope_entries_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, g);
        return cudaGetLastError();
    }
    // from about eight CTAs of four tokens per SM on a CTA takes four: the loads of a token then run
    // beside the arithmetic of the one before; few tokens' heads are spread over the SMs
    g.tokens = a.q.tokens >= kRopeTokens * 8 * sms ? kRopeTokens : 1;
    const int64_t most = cdiv(static_cast<int64_t>(g.tokens) * g.line, kRopeThreads);
    const int64_t want = cdiv(2 * sms, a.q.tokens);
    const dim3 grid(static_cast<unsigned>(cdiv(a.q.tokens, g.tokens)),
                    static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
    if (a.interleaved) {
        if (f16)
            rope_cache_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(a, g);
        else
            rope_cache_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(a, g);
    } else {
        if (f16)
            rope_cache_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(a, g);
        else
            rope_cache_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(a, g);
    }
    return cudaGetLastError();
}

}  // namespace sv
