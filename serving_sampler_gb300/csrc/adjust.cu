// sv_adjust_logits: penalties for repeated tokens, biases and grammar masks on the
// rows of a verify step.
//
// A CTA takes a slice of one request's vocabulary for a few of its rows.  It counts the
// request's tokens that fall into the slice in shared memory (a word an id: seen, times
// in the output, and the head of a chain of the drafts with that id), and lists the ids
// that any rule meets.  Then the rows stream through as masked copies, and the listed ids
// are computed once more and written over them.  In place the copy is left out: rows
// without a mask cost their listed ids alone.
//
// Counts are whole numbers, so the order in which threads meet the tokens changes nothing.
#include <algorithm>
#include <cuda_bf16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kAdjThreads = 512;
constexpr int kAdjChunk = 1024;  // ids that a warp streams at a time
constexpr int kAdjSlice = 8192;  // most ids of a slice
constexpr int kAdjEdge = 8;      // ids before a slice that a row which starts within a vector needs

// a word of the table: bit 31 seen, bits 19 .. 30 the head of the chain (0: none), bits 0 .. 18 the count
constexpr uint32_t kAdjSeen = 1u << 31, kAdjHeadShift = 19, kAdjHead = 0xFFFu << kAdjHeadShift,
                   kAdjCount = (1u << kAdjHeadShift) - 1;
static_assert(SV_MAX_HISTORY <= (1 << kAdjHeadShift) - 1, "a count must not reach the chain's head");
static_assert(SV_MAX_BRANCHES * SV_MAX_K < (1 << 12), "a draft's number must fit the head");

struct AdjustGeom {
    int32_t slice, slices;  // ids of a slice (a power of two), slices of a row
    int32_t rows, groups;   // rows of a request, thread blocks that share them
    int32_t drafts;         // branches * k
};

__host__ __device__ inline size_t table_bytes(const AdjustGeom& g, bool biased)
{
    const size_t ids = g.slice + kAdjEdge;
    return ids * 4 * (biased ? 2 : 1) + (ids / 32 + 1) * 4 + ids * 2 + static_cast<size_t>(g.drafts) * 2;
}

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v)
{
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
template <>
__device__ __forceinline__ float widen<uint32_t>(uint32_t v)
{
    return __uint_as_float(v);
}
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v)
{
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
template <>
__device__ __forceinline__ uint32_t narrow<uint32_t>(float v)
{
    return __float_as_uint(v);
}
template <typename T>
constexpr T kNegInf = static_cast<T>(sizeof(T) == 2 ? 0xFF80u : 0xFF800000u);

// Whether each of the eight ids from x on is allowed, as bits.  x >= 0; bits behind the mask's end are 0.
__device__ __forceinline__ uint32_t allowed8(const uint8_t* mask, int32_t mask_bytes, int32_t x)
{
    const int32_t at = x >> 3, shift = x & 7;
    uint32_t m = mask[at];
    if (shift != 0 && at + 1 < mask_bytes) m |= static_cast<uint32_t>(mask[at + 1]) << 8;
    return (m >> shift) & 0xFFu;
}

// Eight entries with those not allowed set to -inf.
__device__ __forceinline__ void mask8(uint4 (&v)[1], uint32_t m)
{
    uint32_t* w = reinterpret_cast<uint32_t*>(&v[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = (m >> (2 * i)) & 3u;
        const uint32_t keep = ((two | (two << 15)) & 0x00010001u) * 0xFFFFu;
        w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
    }
}
__device__ __forceinline__ void mask8(uint4 (&v)[2], uint32_t m)
{
    uint32_t* w = reinterpret_cast<uint32_t*>(&v[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (m >> i) & 1u ? w[i] : 0xFF800000u;
}

// T: uint16_t for bf16 rows, uint32_t for fp32 rows
template <typename T>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const __grid_constant__ AdjustArgs a, const AdjustGeom g)
{
    constexpr int kVecs = sizeof(T) / 2;  // 16-byte vectors of eight entries
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ int32_t s_listed;
    const sv_logit_rules& u = a.rules;
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t ids = g.slice + kAdjEdge, V = a.in.width;
    const bool biased = u.bias_entries > 0;
    uint32_t* s_tab = s_mem;
    uint32_t* s_bias = s_tab + ids;  // 1 + the last entry of the id's bias, 0 for none
    uint32_t* s_bits = s_bias + (biased ? ids : 0);
    uint16_t* s_list = reinterpret_cast<uint16_t*>(s_bits + ids / 32 + 1);
    uint16_t* s_next = s_list + ids;

    uint32_t block = blockIdx.x;
    const int32_t group = static_cast<int32_t>(block % g.groups);
    block /= g.groups;
    const int32_t s = static_cast<int32_t>(block % g.slices), r = static_cast<int32_t>(block / g.slices);
    const int32_t s0 = s * g.slice, base = s0 - kAdjEdge;  // id of the table's first entry

    for (int i = tid; i < ids; i += kAdjThreads) {
        s_tab[i] = 0;
        if (biased) s_bias[i] = 0;
    }
    for (int i = tid; i < ids / 32 + 1; i += kAdjThreads) s_bits[i] = 0;
    if (tid == 0) s_listed = 0;

    // what the request asks for
    uint32_t st = 0;
    int32_t len = 0, prompt = 0, b0 = 0, b1 = 0;
    if (u.history != nullptr) {
        const int32_t given = u.history_len[r];
        len = min(max(given, 0), u.history_width);
        const int32_t p = u.prompt_len != nullptr ? u.prompt_len[r] : 0;
        prompt = min(max(p, 0), len);
        if (len != given || prompt != p) st |= SV_ST_BAD_LENGTH;
    }
    if (biased) {
        const int32_t x = u.bias_start[r], y = u.bias_start[r + 1];
        b0 = min(max(x, 0), u.bias_entries);
        b1 = min(max(y, b0), u.bias_entries);
        if (b0 != x || b1 != y) st |= SV_ST_BAD_LENGTH;
    }
    float rep = u.repetition != nullptr ? u.repetition[r] : 1.0f;
    float pres = u.presence != nullptr ? u.presence[r] : 0.0f;
    float freq = u.frequency != nullptr ? u.frequency[r] : 0.0f;
    if (!(rep > 0.0f) || isinf(rep)) {
        rep = 1.0f;
        st |= SV_ST_BAD_PENALTY;
    }
    if (!isfinite(pres)) {
        pres = 0.0f;
        st |= SV_ST_BAD_PENALTY;
    }
    if (!isfinite(freq)) {
        freq = 0.0f;
        st |= SV_ST_BAD_PENALTY;
    }
    __syncthreads();

    // The slice's entry of a token (-1: outside), noted in the list when it is the first to meet it.
    bool outside = false;
    auto meet = [&](int32_t x) -> int32_t {
        if (static_cast<uint32_t>(x) >= static_cast<uint32_t>(V)) {
            outside = true;
            return -1;
        }
        const int32_t l = x - base;
        if (l < 0 || l >= ids) return -1;
        const uint32_t bit = 1u << (l & 31);
        if ((atomicOr(&s_bits[l >> 5], bit) & bit) == 0) s_list[atomicAdd(&s_listed, 1)] = static_cast<uint16_t>(l);
        return l;
    };
    const int32_t* history = u.history + static_cast<int64_t>(r) * u.history_width;
    for (int32_t i = tid; i < len; i += kAdjThreads) {
        const int32_t l = meet(history[i]);
        if (l < 0) continue;
        if (i >= prompt)
            atomicAdd(&s_tab[l], 1u);
        else
            atomicOr(&s_tab[l], kAdjSeen);
    }
    for (int32_t i = tid; i < g.drafts; i += kAdjThreads) {
        const int32_t l = meet(a.draft[static_cast<int64_t>(r) * g.drafts + i]);
        if (l < 0) continue;
        uint32_t old = s_tab[l], was;
        do {
            was = old;
            s_next[i] = static_cast<uint16_t>((was & kAdjHead) >> kAdjHeadShift);
            old = atomicCAS(&s_tab[l], was, (was & ~kAdjHead) | (static_cast<uint32_t>(i + 1) << kAdjHeadShift));
        } while (old != was);
    }
    for (int32_t i = b0 + tid; i < b1; i += kAdjThreads) {
        const int32_t l = meet(u.bias_id[i]);
        if (l >= 0) atomicMax(&s_bias[l], static_cast<uint32_t>(i) + 1);
    }
    const int32_t row0 = static_cast<int32_t>(static_cast<int64_t>(g.rows) * group / g.groups);
    const int32_t rows = static_cast<int32_t>(static_cast<int64_t>(g.rows) * (group + 1) / g.groups) - row0;
    const int64_t first = static_cast<int64_t>(r) * g.rows + row0;
    if (s == 0 && group == 0 && a.status != nullptr) {
        bool over = false;
        if (u.mask != nullptr && u.mask_row != nullptr)
            for (int32_t i = tid; i < g.rows; i += kAdjThreads)
                over = over || u.mask_row[static_cast<int64_t>(r) * g.rows + i] >= u.masks;
        if (__syncthreads_or(outside)) st |= SV_ST_TOKEN_RANGE;
        if (__syncthreads_or(over)) st |= SV_ST_BAD_MASK;
        if (tid == 0) a.status[r] = static_cast<int32_t>(st);
    }
    __syncthreads();

    // a row's entries, its mask (or NULL), and how many entries its start lies behind a 16-byte
    // boundary (-1: differently so in the two matrices)
    auto row_of = [&](int32_t j, const T*& in, T*& out, const uint8_t*& mask) -> int32_t {
        in = reinterpret_cast<const T*>(a.in.data) + (first + j) * a.in.stride;
        out = reinterpret_cast<T*>(const_cast<char*>(a.out.data)) + (first + j) * a.out.stride;
        mask = nullptr;
        if (u.mask != nullptr) {
            const int64_t i = u.mask_row != nullptr ? u.mask_row[first + j] : first + j;
            if (i >= 0 && i < u.masks) mask = reinterpret_cast<const uint8_t*>(u.mask + i * u.mask_words);
        }
        const uint32_t x = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(in)) & 15u,
                       y = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) & 15u;
        return x == y ? static_cast<int32_t>(x / sizeof(T)) : -1;
    };
    const bool in_place = a.in.data == a.out.data;
    const int32_t mask_bytes = 4 * u.mask_words;

    if (!in_place || u.mask != nullptr) {
        const int32_t per_row = g.slice / kAdjChunk;
        for (int32_t c = tid / 32; c < rows * per_row; c += kAdjThreads / 32) {
            const T* in;
            T* out;
            const uint8_t* mask;
            const int32_t j = c / per_row, shift = row_of(j, in, out, mask);
            const int32_t x0 = s0 + (c - j * per_row) * kAdjChunk - max(shift, 0);
            if (x0 >= V || (in_place && mask == nullptr)) continue;
            if (shift < 0) {
                for (int32_t x = x0 + lane; x < min(x0 + kAdjChunk, V); x += 32) {
                    const bool ok = mask == nullptr || ((mask[x >> 3] >> (x & 7)) & 1);
                    out[x] = ok ? in[x] : kNegInf<T>;
                }
                continue;
            }
            uint32_t m[4];
            uint4 v[4][kVecs];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int32_t x = x0 + q * 256 + lane * 8;
                const bool whole = x >= 0 && x + 8 <= V;
                m[q] = 0xFFu;
                if (!whole) continue;
                if (mask != nullptr) m[q] = allowed8(mask, mask_bytes, x);
                if (!in_place || (m[q] != 0u && m[q] != 0xFFu))
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) v[q][i] = reinterpret_cast<const uint4*>(in + x)[i];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int32_t x = x0 + q * 256 + lane * 8;
                if (x >= 0 && x + 8 <= V) {
                    if (in_place && m[q] == 0xFFu) continue;
                    if (m[q] != 0xFFu) mask8(v[q], m[q]);
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(out + x)[i] = v[q][i];
                } else {
                    for (int32_t y = max(x, 0); y < min(x + 8, V); ++y) {
                        const bool ok = mask == nullptr || ((mask[y >> 3] >> (y & 7)) & 1);
                        if (!in_place || !ok) out[y] = ok ? in[y] : kNegInf<T>;
                    }
                }
            }
        }
        __syncthreads();
    }

    // the ids that a rule meets
    const int32_t listed = s_listed;
    for (int32_t p = tid; p < rows * listed; p += kAdjThreads) {
        const int32_t j = p / listed, l = s_list[p - j * listed], x = base + l;
        const T* in;
        T* out;
        const uint8_t* mask;
        const int32_t shift = max(row_of(j, in, out, mask), 0);
        if (x < s0 - shift || x >= s0 + g.slice - shift) continue;  // another slice's in this row
        if (mask != nullptr && !((mask[x >> 3] >> (x & 7)) & 1)) continue;
        // the drafts before the row: the first i + 1 of branch b, for row 1 + b * k + i
        const int32_t row = row0 + j;
        int32_t lo = 0, hi = 0;
        if (row > 0) {
            lo = (row - 1) / a.k * a.k;
            hi = row;
        }
        const uint32_t word = s_tab[l];
        uint32_t count = word & kAdjCount;
        for (uint32_t e = (word & kAdjHead) >> kAdjHeadShift; e != 0; e = s_next[e - 1])
            count += static_cast<int32_t>(e) > lo && static_cast<int32_t>(e) <= hi;
        const uint32_t entry = biased ? s_bias[l] : 0u;
        const bool seen = (word & kAdjSeen) != 0 || count != 0;
        if (!seen && entry == 0) continue;
        float z = widen<T>(in[x]);
        if (seen) z = z > 0.0f ? z / rep : z * rep;
        if (count != 0) z -= pres + freq * static_cast<float>(count);
        if (entry != 0) z += u.bias_value[entry - 1];
        out[x] = narrow<T>(z);
    }
}

AdjustGeom geom_of(const AdjustArgs& a)
{
    const int sms = std::max(1, device_sm_count());
    AdjustGeom g{};
    g.drafts = a.branches * a.k;
    g.rows = 1 + g.drafts;
    auto slices = [&](int64_t n) { return (static_cast<int64_t>(a.in.width) + kAdjEdge - 1 + n - 1) / n; };
    g.slice = kAdjSlice;
    while (g.slice > kAdjChunk && a.R * slices(g.slice) < 2 * sms) g.slice /= 2;
    g.slices = static_cast<int32_t>(slices(g.slice));
    const int64_t blocks = static_cast<int64_t>(a.R) * g.slices;
    g.groups = static_cast<int32_t>(std::min<int64_t>(g.rows, std::max<int64_t>(1, 4 * sms / blocks)));
    return g;
}

}  // namespace

bool adjust_fits(const AdjustArgs& a)
{
    const AdjustGeom g = geom_of(a);
    return static_cast<int64_t>(a.R) * g.slices * g.groups <= INT32_MAX;
}

cudaError_t launch_adjust_logits(const AdjustArgs& a, cudaStream_t stream)
{
    const AdjustGeom g = geom_of(a);
    const size_t bytes = table_bytes(g, a.rules.bias_entries > 0);
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.R) * g.slices * g.groups);
    auto* kernel = a.in.dtype == SV_BF16 ? adjust_kernel<uint16_t> : adjust_kernel<uint32_t>;
    if (cudaError_t e = allow_shared(kernel, static_cast<int>(bytes))) return e;
    kernel<<<blocks, kAdjThreads, bytes, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
