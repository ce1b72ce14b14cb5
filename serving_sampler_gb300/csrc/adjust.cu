// sv_adjust_logits: penalties for repeated tokens, biases and grammar masks on the
// rows of a verify step.
//
// A CTA takes a slice of one request's vocabulary for a few of its rows.  Half of its warps
// stream the rows through as masked copies.  The others meanwhile count the request's tokens
// that fall into the slice in shared memory (a word an id: seen, times in the output, and
// the head of a chain of the drafts with that id), list the ids that any rule meets, and
// compute those ids' entries of every row, which are written over the copies at the end.
// In place the copy is left out: rows without a mask cost their listed ids alone.
//
// Counts are whole numbers, so the order in which threads meet the tokens changes nothing.
#include <algorithm>
#include <cuda_bf16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kAdjThreads = 512;
constexpr int kAdjBuilders = 256;  // threads that count, list and compute while the others copy
constexpr int kAdjChunk = 1024;    // ids that a warp copies at a time
constexpr int kAdjSlice = 8192;    // most ids of a slice
constexpr int kAdjEdge = 8;        // ids before a slice that a row which starts within a vector needs
constexpr int kAdjKept = 4096;     // computed entries that wait for the copies
constexpr int kAdjBatch = 8;       // tokens that a thread loads before it counts them

// a word of the table: bit 31 seen, bits 19 .. 30 the head of the chain (0: none), bits 0 .. 18 the count
constexpr uint32_t kAdjSeen = 1u << 31, kAdjHeadShift = 19, kAdjHead = 0xFFFu << kAdjHeadShift,
                   kAdjCount = (1u << kAdjHeadShift) - 1;
static_assert(SV_MAX_HISTORY <= (1 << kAdjHeadShift) - 1, "a count must not reach the chain's head");
static_assert(SV_MAX_BRANCHES * SV_MAX_K < (1 << 12), "a draft's number must fit the head");

struct AdjustGeom {
    int32_t slice, slices;  // ids of a slice (a power of two), slices of a row
    int32_t rows, groups;   // rows of a request, thread blocks that share them
    int32_t most_rows;      // of a thread block
    int32_t drafts;         // branches * k
};

// The parts of a CTA's shared memory, in 32-bit words.
struct AdjustLayout {
    int32_t bias, bits, kept, mask, list, next, bytes;  // the table lies first; list and next hold 16 bits each
};
__host__ __device__ inline AdjustLayout layout_of(const AdjustGeom& g, bool biased, int esize)
{
    const int32_t ids = g.slice + kAdjEdge;
    AdjustLayout l;
    l.bias = ids;
    l.bits = l.bias + (biased ? ids : 0);
    l.kept = l.bits + ids / 32 + 1;
    l.mask = l.kept + kAdjKept * esize / 4;
    l.list = l.mask + g.most_rows;
    l.next = l.list + ids / 2;
    l.bytes = 4 * (l.next + (g.drafts + 1) / 2);
    return l;
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

// Whether each of the N ids from x on is allowed, as bits.  x >= 0; bits behind the mask's end are 0.
template <int N>
__device__ __forceinline__ uint32_t allowed(const uint8_t* mask, int32_t mask_bytes, int32_t x)
{
    const int32_t at = x >> 3, shift = x & 7;
    uint32_t m = mask[at];
    if (shift > 8 - N && at + 1 < mask_bytes) m |= static_cast<uint32_t>(mask[at + 1]) << 8;
    return (m >> shift) & ((1u << N) - 1);
}

// A vector's entries, those not allowed set to -inf.
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 v, uint32_t m)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 2) {
            const uint32_t two = (m >> (2 * i)) & 3u;
            const uint32_t keep = ((two | (two << 15)) & 0x00010001u) * 0xFFFFu;
            w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
        } else {
            w[i] = (m >> i) & 1u ? w[i] : 0xFF800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void builders_sync(int threads)
{
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// T: uint16_t for bf16 rows, uint32_t for fp32 rows
template <typename T>
__global__ void __launch_bounds__(kAdjThreads, 2) adjust_kernel(const __grid_constant__ AdjustArgs a, const AdjustGeom g)
{
    constexpr int kPer = 16 / sizeof(T);                // entries of a vector
    constexpr int kVecs = kAdjChunk / (32 * kPer);      // vectors that a lane holds
    constexpr uint32_t kAll = (1u << kPer) - 1;
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ int32_t s_listed, s_chunk;
    const sv_logit_rules& u = a.rules;
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t ids = g.slice + kAdjEdge, V = a.in.width;
    const bool biased = u.bias_entries > 0;
    const AdjustLayout at = layout_of(g, biased, sizeof(T));
    uint32_t* s_tab = s_mem;
    uint32_t* s_bias = s_mem + at.bias;  // 1 + the last entry of the id's bias, 0 for none
    uint32_t* s_bits = s_mem + at.bits;
    T* s_kept = reinterpret_cast<T*>(s_mem + at.kept);
    int32_t* s_mask = reinterpret_cast<int32_t*>(s_mem + at.mask);  // each row's mask, -1 for none
    uint16_t* s_list = reinterpret_cast<uint16_t*>(s_mem + at.list);
    uint16_t* s_next = reinterpret_cast<uint16_t*>(s_mem + at.next);

    uint32_t block = blockIdx.x;
    const int32_t group = static_cast<int32_t>(block % g.groups);
    block /= g.groups;
    const int32_t s = static_cast<int32_t>(block % g.slices), r = static_cast<int32_t>(block / g.slices);
    const int32_t s0 = s * g.slice, base = s0 - kAdjEdge;  // id of the table's first entry
    const int32_t row0 = static_cast<int32_t>(static_cast<int64_t>(g.rows) * group / g.groups);
    const int32_t rows = static_cast<int32_t>(static_cast<int64_t>(g.rows) * (group + 1) / g.groups) - row0;
    const int64_t first = static_cast<int64_t>(r) * g.rows + row0;
    const bool in_place = a.in.data == a.out.data;
    const bool copies = !in_place || u.mask != nullptr;
    const int32_t mask_bytes = 4 * u.mask_words;

    for (int i = tid; i < at.kept / 4 + 1; i += kAdjThreads) reinterpret_cast<uint4*>(s_mem)[i] = make_uint4(0, 0, 0, 0);
    for (int j = tid; j < rows; j += kAdjThreads) {
        int64_t i = -1;
        if (u.mask != nullptr) i = u.mask_row != nullptr ? u.mask_row[first + j] : first + j;
        s_mask[j] = i >= 0 && i < u.masks ? static_cast<int32_t>(i) : -1;
    }
    if (tid == 0) s_listed = s_chunk = 0;
    __syncthreads();

    // a row's entries, its mask (or NULL), and how many entries its start lies behind a 16-byte
    // boundary (-1: differently so in the two matrices)
    auto row_of = [&](int32_t j, const T*& in, T*& out, const uint8_t*& mask) -> int32_t {
        in = reinterpret_cast<const T*>(a.in.data) + (first + j) * a.in.stride;
        out = reinterpret_cast<T*>(const_cast<char*>(a.out.data)) + (first + j) * a.out.stride;
        const int32_t i = s_mask[j];
        mask = i < 0 ? nullptr : reinterpret_cast<const uint8_t*>(u.mask + static_cast<int64_t>(i) * u.mask_words);
        const uint32_t x = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(in)) & 15u,
                       y = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out)) & 15u;
        return x == y ? static_cast<int32_t>(x / sizeof(T)) : -1;
    };
    // Entry p of the listed ids' entries, row by row: its id and place, or false where it is another slice's.
    float rep = 1.0f, pres = 0.0f, freq = 0.0f;
    auto place_of = [&](int32_t p, int32_t listed, int32_t& j, int32_t& l, const T*& in, T*& out, const uint8_t*& mask) {
        j = p / listed;
        l = s_list[p - j * listed];
        const int32_t shift = max(row_of(j, in, out, mask), 0), x = base + l;
        return x >= s0 - shift && x < s0 + g.slice - shift;
    };
    // The adjusted entry of the table's id l in row j.
    auto entry_of = [&](int32_t j, int32_t l, const T* in, const uint8_t* mask) -> T {
        const int32_t x = base + l;
        const T raw = in[x];
        if (mask != nullptr && !((mask[x >> 3] >> (x & 7)) & 1)) return kNegInf<T>;
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
        if (!seen && entry == 0) return raw;
        float z = widen<T>(raw);
        if (seen) z = z > 0.0f ? z / rep : z * rep;
        if (count != 0) z -= pres + freq * static_cast<float>(count);
        if (entry != 0) z += u.bias_value[entry - 1];
        return narrow<T>(z);
    };

    // what the request asks for
    uint32_t st = 0;
    if (u.repetition != nullptr) rep = u.repetition[r];
    if (u.presence != nullptr) pres = u.presence[r];
    if (u.frequency != nullptr) freq = u.frequency[r];
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

    const int builders = copies ? kAdjBuilders : kAdjThreads;
    if (tid < builders) {
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
        // The slice's entry of a token (-1: outside), noted in the list by the first to meet it.
        auto meet = [&](int32_t x) -> int32_t {
            if (static_cast<uint32_t>(x) >= static_cast<uint32_t>(V)) {
                st |= SV_ST_TOKEN_RANGE;
                return -1;
            }
            const int32_t l = x - base;
            if (l < 0 || l >= ids) return -1;
            const uint32_t bit = 1u << (l & 31);
            if ((atomicOr(&s_bits[l >> 5], bit) & bit) == 0) s_list[atomicAdd(&s_listed, 1)] = static_cast<uint16_t>(l);
            return l;
        };
        const int32_t* history = u.history + static_cast<int64_t>(r) * u.history_width;
        for (int32_t i0 = tid; i0 < len; i0 += builders * kAdjBatch) {
            int32_t token[kAdjBatch];
#pragma unroll
            for (int q = 0; q < kAdjBatch; ++q)
                if (i0 + q * builders < len) token[q] = history[i0 + q * builders];
#pragma unroll
            for (int q = 0; q < kAdjBatch; ++q) {
                const int32_t i = i0 + q * builders;
                const int32_t l = i < len ? meet(token[q]) : -1;
                if (l < 0) continue;
                if (i >= prompt)
                    atomicAdd(&s_tab[l], 1u);
                else
                    atomicOr(&s_tab[l], kAdjSeen);
            }
        }
        for (int32_t i = tid; i < g.drafts; i += builders) {
            const int32_t l = meet(a.draft[static_cast<int64_t>(r) * g.drafts + i]);
            if (l < 0) continue;
            uint32_t old = s_tab[l], was;
            do {
                was = old;
                s_next[i] = static_cast<uint16_t>((was & kAdjHead) >> kAdjHeadShift);
                old = atomicCAS(&s_tab[l], was, (was & ~kAdjHead) | (static_cast<uint32_t>(i + 1) << kAdjHeadShift));
            } while (old != was);
        }
        for (int32_t i = b0 + tid; i < b1; i += builders) {
            const int32_t l = meet(u.bias_id[i]);
            if (l >= 0) atomicMax(&s_bias[l], static_cast<uint32_t>(i) + 1);
        }
        builders_sync(builders);
        const int32_t listed = s_listed, kept = min(rows * listed, kAdjKept);
        for (int32_t p = tid; p < kept; p += builders) {
            int32_t j, l;
            const T* in;
            T* out;
            const uint8_t* mask;
            if (place_of(p, listed, j, l, in, out, mask)) s_kept[p] = entry_of(j, l, in, mask);
        }
    }

    if (copies) {
        const int32_t per_row = g.slice / kAdjChunk;
        for (;;) {
            int32_t c = 0;
            if (lane == 0) c = atomicAdd(&s_chunk, 1);
            c = __shfl_sync(0xFFFFFFFFu, c, 0);
            if (c >= rows * per_row) break;
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
            uint32_t m[kVecs];
            uint4 v[kVecs];
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int32_t x = x0 + (q * 32 + lane) * kPer;
                const bool whole = x >= 0 && x + kPer <= V;
                m[q] = whole && mask != nullptr ? allowed<kPer>(mask, mask_bytes, x) : kAll;
                if (whole && (!in_place || (m[q] != 0u && m[q] != kAll))) v[q] = *reinterpret_cast<const uint4*>(in + x);
            }
#pragma unroll
            for (int q = 0; q < kVecs; ++q) {
                const int32_t x = x0 + (q * 32 + lane) * kPer;
                if (x >= 0 && x + kPer <= V) {
                    if (in_place && m[q] == kAll) continue;
                    *reinterpret_cast<uint4*>(out + x) = m[q] != kAll ? masked<T>(v[q], m[q]) : v[q];
                } else {
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y) {
                        const bool ok = mask == nullptr || ((mask[y >> 3] >> (y & 7)) & 1);
                        if (!in_place || !ok) out[y] = ok ? in[y] : kNegInf<T>;
                    }
                }
            }
        }
    }
    if (s == 0 && group == 0 && a.status != nullptr) {
        if (u.mask != nullptr && u.mask_row != nullptr)
            for (int32_t i = tid; i < g.rows; i += kAdjThreads)
                if (u.mask_row[static_cast<int64_t>(r) * g.rows + i] >= u.masks) st |= SV_ST_BAD_MASK;
        // every thread but those that count leaves some bits unset
        st = (__syncthreads_or(st & SV_ST_TOKEN_RANGE) ? SV_ST_TOKEN_RANGE : 0u) |
             (__syncthreads_or(st & SV_ST_BAD_MASK) ? SV_ST_BAD_MASK : 0u) | (st & (SV_ST_BAD_LENGTH | SV_ST_BAD_PENALTY));
        if (tid == 0) a.status[r] = static_cast<int32_t>(st);
    }
    __syncthreads();

    // the computed entries over the copies
    const int32_t listed = s_listed;
    for (int32_t p = tid; p < rows * listed; p += kAdjThreads) {
        int32_t j, l;
        const T* in;
        T* out;
        const uint8_t* mask;
        if (!place_of(p, listed, j, l, in, out, mask)) continue;
        out[base + l] = p < kAdjKept ? s_kept[p] : entry_of(j, l, in, mask);
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
    g.most_rows = (g.rows + g.groups - 1) / g.groups;
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
    const int bytes = layout_of(g, a.rules.bias_entries > 0, a.in.esize).bytes;
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.R) * g.slices * g.groups);
    auto* kernel = a.in.dtype == SV_BF16 ? adjust_kernel<uint16_t> : adjust_kernel<uint32_t>;
    if (cudaError_t e = allow_shared(kernel, bytes)) return e;
    kernel<<<blocks, kAdjThreads, bytes, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
