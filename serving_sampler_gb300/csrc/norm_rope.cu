// sv_norm_rope_cache: an RMS norm of every q and k head, rotary positions, k and v
// written into the paged cache, one read and one write of every head.
//
// y = x * (mean(x^2) + eps)^(-1/2) * w, then pairs of y turn as in rope.cu.  The sum of
// squares needs a whole head before its first entry can be written, so a head belongs to
// the lanes that hold its vectors two by two (the same two of every head: the halves of
// eight pairs, or neighbours), and the sum is taken by exchanges among them.  Arithmetic
// is on pairs of fp32 values.
//
// Bound by bytes where there are many: 51.0 us for the 284 MB of 15,420 tokens, 32 + 8 heads of 96, 5.6 TB/s, 0.82 of
// a copy's rate (62 for 379 MB with heads of 128, 0.90); 14.7 us for the 77 MB of 4,160 tokens, 28 + 4 heads of 128;
// 3.7 us, a launch, for one token.  With 8 lanes to a head of 96, of which two had nothing, tables read across banks
// and single values the first two took 64 and 23.  It issues 38.6 M warp instructions in the first, 0.67 of what it
// could; a table of the heads' places saves a fifth of them and no time.
#include <algorithm>

#include "sv_internal.h"
#include "sv_rope.cuh"

namespace sv {
namespace {

constexpr int kNormTokens = 4;  // most tokens of a CTA

struct NormGeom {
    int32_t half;    // rotated pairs
    int32_t rows;    // q heads, then k heads, then v heads
    int32_t items;   // lanes that a head's vectors of 8 entries fill, two each
    int32_t tokens;  // of a CTA
    float by_dim;    // 1 / head_dim
};

__device__ __forceinline__ float weight_at(const void* w, int32_t dtype, int i)
{
    if (w == nullptr) return 1.0f;
    if (dtype == SV_F32) return static_cast<const float*>(w)[i];
    if (dtype == SV_F16) return __half2float(static_cast<const __half*>(w)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Two fp32 values times a factor, and the two 16-bit entries of a word as fp32.
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }
template <bool F16>
__device__ __forceinline__ uint64_t wide2(uint32_t w)
{
    const float2 v = unpack2<F16>(w);
    return pack2(v.x, v.y);
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(uint64_t v)
{
    float x, y;
    unpack2(v, x, y);
    return pack2<F16>(x, y);
}

// A vector of E 16-bit entries.
template <int E>
struct Packed {
    uint32_t w[E / 2];
};
template <int E>
__device__ __forceinline__ Packed<E> load_packed(const void* p)
{
    Packed<E> v;
    if constexpr (E == 8) {
        const uint4 x = *static_cast<const uint4*>(p);
        v.w[0] = x.x, v.w[1] = x.y, v.w[2] = x.z, v.w[3] = x.w;
    } else if constexpr (E == 4) {
        const uint2 x = *static_cast<const uint2*>(p);
        v.w[0] = x.x, v.w[1] = x.y;
    } else {
        v.w[0] = *static_cast<const uint32_t*>(p);
    }
    return v;
}
template <int E>
__device__ __forceinline__ void store_packed(void* p, const Packed<E>& v)
{
    if constexpr (E == 8)
        *static_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    else if constexpr (E == 4)
        *static_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
    else
        *static_cast<uint32_t*>(p) = v.w[0];
}

// SIDE: as in rope.cu.  ITEMS: lanes of a head, 32 / ITEMS heads to a warp.  E: entries of a vector, of which the
// distance between a pair's halves is a multiple (8 where pairs lie side by side).
template <bool F16, bool SIDE, int ITEMS, int E>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs n, const NormGeom g)
{
    constexpr int kHeads = 32 / ITEMS, kGroups = kRopeThreads / 32 * kHeads, kParts = E / 2;
    const RopeArgs& a = n.rope;
    // What a lane reads of the tables lies 16 bytes beside what the next lane reads: [part][lane of the head].
    __shared__ __align__(16) float4 s_cs[kNormTokens][kParts][ITEMS];  // cosine and sine of two pairs
    __shared__ __align__(16) float4 s_w[2][kParts][ITEMS];             // four entries' weights for q, for k
    __shared__ int64_t s_at[kNormTokens];
    const int tid = threadIdx.x, lane = tid & 31;
    const bool whole = lane < kHeads * ITEMS;  // the last lanes of a warp may have no head
    const int j = whole ? lane % ITEMS : 0, group = whole ? tid / 32 * kHeads + lane / ITEMS : 0;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * g.tokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(g.tokens), a.q.tokens - t0));
    const int Hq = a.q.heads, Hk = a.cache.kv_heads, D = a.cache.head_dim;
    const int step = kGroups * gridDim.y;

    // the two vectors of a lane, and whether pairs turn in them
    const int cut = g.half / E, vecs = D / E;
    auto vectors_of = [&](int j, int& va, int& vb) -> bool {
        va = 2 * j;
        vb = 2 * j + 1;
        if (SIDE) return 8 * j < g.half;
        if (j >= cut) return false;
        va = j;
        vb = j + cut;
        return true;
    };
    int va_at, vb_at;
    const bool turns = vectors_of(j, va_at, vb_at), has_a = whole && va_at < vecs, has_b = whole && vb_at < vecs;

    struct Head {
        int token, row;
        __device__ __forceinline__ void settle(int rows)
        {
#pragma unroll 1
            while (row >= rows) {
                row -= rows;
                ++token;
            }
        }
    };
    auto load = [&](const Head& h, Packed<E>& va, Packed<E>& vb) {
        va = vb = Packed<E>{};
        if (h.token >= tokens) return;
        const sv_heads& m = h.row < Hq ? a.q : h.row < Hq + Hk ? a.k : a.v;
        const int r = h.row < Hq ? h.row : h.row < Hq + Hk ? h.row - Hq : h.row - Hq - Hk;
        const uint16_t* src = static_cast<const uint16_t*>(m.data) + (t0 + h.token) * m.token_stride + r * m.head_stride;
        if (has_a) va = load_packed<E>(src + va_at * E);
        if (has_b) vb = load_packed<E>(src + vb_at * E);
    };
    Packed<E> na, nb;  // the next head's vectors, in flight
    Head next{0, static_cast<int>(blockIdx.y) * kGroups + group};
    next.settle(g.rows);
    load(next, na, nb);
    if (tid < tokens) s_at[tid] = slot_offset(a, a.slot[t0 + tid]);
    for (int i = tid; i < 2 * kParts * ITEMS; i += kRopeThreads) {
        const int which = i / (kParts * ITEMS), part = i / ITEMS % kParts, o = i % ITEMS;
        int x, y;
        vectors_of(o, x, y);
        const void* w = which == 0 ? n.q_weight : n.k_weight;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int at = 4 * part + e, entry = at < E ? E * x + at : E * y + at - E;  // of the lane's 2 E
            f[e] = w != nullptr && entry < D ? weight_at(w, n.weight_dtype, entry) : 1.0f;
        }
        s_w[which][part][o] = make_float4(f[0], f[1], f[2], f[3]);
    }
    for (int y = tid; y < tokens * E * ITEMS; y += kRopeThreads) {
        const int i = y / (E * ITEMS), p = y - i * (E * ITEMS);
        // a lane may hold fewer pairs than E: the others pass
        const float2 t = p < g.half ? turn_of(a, a.position[t0 + i], p) : make_float2(1.0f, 0.0f);
        float* to = &s_cs[i][p / 2 % kParts][p / E].x + p % 2 * (SIDE ? 2 : 1);
        to[0] = t.x;             // side by side: cosine, sine of each; else the two cosines, then the two sines
        to[SIDE ? 1 : 2] = t.y;
    }
    __syncthreads();

    // every warp takes the same number of rounds: the exchanges need all of its lanes
    const int total = tokens * g.rows;
    for (int base = static_cast<int>(blockIdx.y) * kGroups; base < total; base += step) {
        Packed<E> va = na, vb = nb;
        const Head h = next;
        next.row += step;
        next.settle(g.rows);
        load(next, na, nb);
        uint64_t f[E], sums = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            f[e] = wide2<F16>(e < kParts ? va.w[e % kParts] : vb.w[e % kParts]);
            sums = fma2(f[e], f[e], sums);
        }
        float lo, hi;
        unpack2(sums, lo, hi);
        float sum = lo + hi;
        if ((ITEMS & (ITEMS - 1)) == 0) {
#pragma unroll
            for (int d = 1; d < ITEMS; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        } else {
            // the head's lanes in the same order for each of them
            float all = 0.0f;
#pragma unroll
            for (int d = 0; d < ITEMS; ++d) all += __shfl_sync(0xFFFFFFFFu, sum, lane - j + d);
            sum = all;
        }
        if (!whole || h.token >= tokens) continue;
        if (h.row < Hq + Hk) {
            const uint64_t scale = both(rsqrtf(sum * g.by_dim + n.eps));
            const int which = h.row < Hq ? 0 : 1;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const float4 u = s_w[which][part][j];
                f[2 * part] = mul2(f[2 * part], mul2(pack2(u.x, u.y), scale));
                f[2 * part + 1] = mul2(f[2 * part + 1], mul2(pack2(u.z, u.w), scale));
            }
            if (turns) {
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    const float4 t = s_cs[h.token][part][j];
                    if (SIDE) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float c = e == 0 ? t.x : t.z, sn = e == 0 ? t.y : t.w;
                            float x, y;
                            unpack2(f[2 * part + e], x, y);
                            f[2 * part + e] = fma2(pack2(y, x), pack2(-sn, sn), mul2(f[2 * part + e], both(c)));
                        }
                    } else {
                        const uint64_t c = pack2(t.x, t.y), sn = pack2(t.z, t.w), x = f[part], y = f[kParts + part];
                        f[part] = fma2(y, pack2(-t.z, -t.w), mul2(x, c));
                        f[kParts + part] = fma2(x, sn, mul2(y, c));
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < kParts; ++e) {
                va.w[e] = narrow2<F16>(f[e]);
                vb.w[e] = narrow2<F16>(f[kParts + e]);
            }
        }
        uint16_t* dst;
        if (h.row < Hq) {
            dst = static_cast<uint16_t*>(const_cast<void*>(a.q_out.data)) + (t0 + h.token) * a.q_out.token_stride +
                  h.row * a.q_out.head_stride;
        } else {
            const int64_t at = s_at[h.token];
            if (at < 0) continue;
            const bool key = h.row < Hq + Hk;
            dst = static_cast<uint16_t*>(key ? a.cache.k : a.cache.v) + at + (h.row - (key ? Hq : Hq + Hk)) * a.cache.head_stride;
        }
        if (has_a) store_packed<E>(dst + va_at * E, va);
        if (has_b) store_packed<E>(dst + vb_at * E, vb);
    }
}

// Halves that lie apart by an odd number of entries: a warp takes a head, entry by entry, and
// gets the partners' values by a second read of them; it has read all before it writes any.
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_entries_kernel(const __grid_constant__ NormRopeArgs n,
                                                                         const NormGeom g)
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

template <bool F16, bool SIDE, int ITEMS, int E>
void launch_items(const NormRopeArgs& n, NormGeom& g, cudaStream_t stream)
{
    constexpr int kGroups = kRopeThreads / 32 * (32 / ITEMS);
    const int64_t T = n.rope.q.tokens;
    const int sms = device_sm_count();
    auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    // from 16 tokens per SM on a CTA takes four: 4,160 tokens 14.7 us instead of 17.3; at 8 per SM 10.4 instead of 7.4
    g.tokens = T >= kNormTokens * 4 * sms ? kNormTokens : 1;
    const int64_t most = cdiv(static_cast<int64_t>(g.tokens) * g.rows, kGroups);
    const int64_t want = cdiv(2 * sms, T);
    const dim3 grid(static_cast<unsigned>(cdiv(T, g.tokens)),
                    static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
    norm_rope_kernel<F16, SIDE, ITEMS, E><<<grid, kRopeThreads, 0, stream>>>(n, g);
}

// The lanes that a head's vectors fill, for vectors of 8 entries.
template <bool F16, bool SIDE, int ITEMS>
void launch_eights(const NormRopeArgs& n, NormGeom& g, cudaStream_t stream)
{
    if (g.items == ITEMS)
        launch_items<F16, SIDE, ITEMS, 8>(n, g, stream);
    else if constexpr (ITEMS > 1)
        launch_eights<F16, SIDE, ITEMS - 1>(n, g, stream);
}

// Halves that lie apart by a multiple of 4 or of 2 entries: a power of two of lanes.  4,160 tokens, 28 + 4 heads of 96
// with 24 rotated take 20 us, of 80 with 20 rotated 28, where an entry at a time takes 37 for either.
template <bool F16>
void launch_shorter(const NormRopeArgs& n, NormGeom& g, cudaStream_t stream)
{
    const bool fours = g.half % 4 == 0, small = n.rope.cache.head_dim <= SV_MAX_HEAD_DIM / 2;
    if (fours && small)
        launch_items<F16, false, SV_MAX_HEAD_DIM / 16, 4>(n, g, stream);
    else if (fours)
        launch_items<F16, false, SV_MAX_HEAD_DIM / 8, 4>(n, g, stream);
    else if (small)
        launch_items<F16, false, SV_MAX_HEAD_DIM / 8, 2>(n, g, stream);
    else
        launch_items<F16, false, SV_MAX_HEAD_DIM / 4, 2>(n, g, stream);
}

}  // namespace

cudaError_t launch_norm_rope_cache(const NormRopeArgs& n, cudaStream_t stream)
{
    const RopeArgs& a = n.rope;
    NormGeom g{};
    g.half = a.rot_dim / 2;
    g.rows = a.q.heads + 2 * a.cache.kv_heads;
    g.items = (a.cache.head_dim / 8 + 1) / 2;
    g.by_dim = 1.0f / a.cache.head_dim;
    const int sms = device_sm_count();
    const bool f16 = a.cache.dtype == SV_F16;
    auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    if (!a.interleaved && g.half % 2 != 0) {
        const int64_t most = cdiv(g.rows, kRopeThreads / 32), want = cdiv(8 * sms, a.q.tokens);
        const dim3 grid(static_cast<unsigned>(a.q.tokens), static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))));
        if (f16)
            norm_rope_entries_kernel<true><<<grid, kRopeThreads, 0, stream>>>(n, g);
        else
            norm_rope_entries_kernel<false><<<grid, kRopeThreads, 0, stream>>>(n, g);
        return cudaGetLastError();
    }
    constexpr int kMost = SV_MAX_HEAD_DIM / 16;
    if (a.interleaved) {
        if (f16)
            launch_eights<true, true, kMost>(n, g, stream);
        else
            launch_eights<false, true, kMost>(n, g, stream);
    } else if (g.half % 8 == 0) {
        if (f16)
            launch_eights<true, false, kMost>(n, g, stream);
        else
            launch_eights<false, false, kMost>(n, g, stream);
    } else {
        if (f16)
            launch_shorter<true>(n, g, stream);
        else
            launch_shorter<false>(n, g, stream);
    }
    return cudaGetLastError();
}

}  // namespace sv
