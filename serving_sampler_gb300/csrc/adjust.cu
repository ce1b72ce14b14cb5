// sv_adjust_logits: penalties for repeated tokens, biases and grammar masks on the
// rows of a verify step.
//
// A CTA takes a slice of one request's vocabulary for a few of its rows.  It counts the
// request's tokens that fall into the slice in shared memory (a word an id: seen, times
// in the output, and the head of a chain of the drafts with that id) and lists the ids that
// any rule meets, by regions of the slice.  Then each warp takes regions of rows by itself:
// asynchronous copies bring the next ones into its ring of tiles while it adjusts the listed
// entries of the present one in shared memory and stores it masked.  The first copies are in
// flight while the tokens are counted.
// In place nothing is copied: masked entries are written, listed ones read and written.
//
// Counts are whole numbers, so the order in which threads meet the tokens changes nothing.
#include <algorithm>
#include <cuda_bf16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjVecs = 4;                      // 16-byte vectors of a tile that a lane holds
constexpr int kAdjTile = kAdjVecs * 32 * 16;     // bytes of a tile: a region of a row
constexpr int kAdjStages = 2;                    // tiles of a warp's ring
constexpr int kAdjSlice = 4096;                  // most ids of a slice
constexpr int kAdjEdge = 8;                      // ids before a slice that a row which starts within a vector needs
constexpr int kAdjBatch = 8;                     // tokens that a thread loads before it counts them
constexpr int kAdjMaskWords = kAdjTile / 2 / 32 + 1;  // words of a region's mask

// a word of the table: bit 31 seen, bits 19 .. 30 the head of the chain (0: none), bits 0 .. 18 the count
constexpr uint32_t kAdjSeen = 1u << 31, kAdjHeadShift = 19, kAdjHead = 0xFFFu << kAdjHeadShift,
                   kAdjCount = (1u << kAdjHeadShift) - 1;
static_assert(SV_MAX_HISTORY <= (1 << kAdjHeadShift) - 1, "a count must not reach the chain's head");
static_assert(SV_MAX_BRANCHES * SV_MAX_K < (1 << 12), "a draft's number must fit the head");
static_assert(kAdjSlice / (kAdjTile / 4) <= kAdjWarps, "a warp keeps to one region, and a region has a warp");
static_assert(kAdjMaskWords >= 33, "a warp brings 33 words of a mask");

struct AdjustGeom {
    int32_t slice, slices;  // ids of a slice (a power of two), slices of a row
    int32_t region_shift;   // log2 of a slice's regions, at most kAdjWarps
    int32_t rows, groups;   // rows of a request, thread blocks that share them
    int32_t most_rows;      // of a thread block
    int32_t drafts;         // branches * k
    int32_t bias_bits;      // of an id's word in the table of biases: 0 without biases, 16 where their numbers fit, else 32
};

// The parts of a CTA's shared memory, in 32-bit words; the tiles lie first.
struct AdjustLayout {
    int32_t mask, tab, bias, row, list, next, bytes;  // list and next hold 16 bits each
};
__host__ __device__ inline AdjustLayout layout_of(const AdjustGeom& g, bool tiles)
{
    const int32_t ids = g.slice + kAdjEdge;
    AdjustLayout l;
    l.mask = tiles ? kAdjWarps * kAdjStages * kAdjTile / 4 : 0;
    l.tab = l.mask + (tiles ? (kAdjWarps * kAdjStages * kAdjMaskWords + 3) / 4 * 4 : 0);
    l.bias = l.tab + ids;
    l.row = l.bias + ids * g.bias_bits / 32;
    l.list = l.row + 2 * g.most_rows;
    l.next = l.list + (g.slice + (kAdjEdge << g.region_shift)) / 2;
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

__device__ __forceinline__ bool allowed(const uint32_t* mask, int32_t x)
{
    return mask == nullptr || ((mask[x >> 5] >> (x & 31)) & 1u);
}

// The signs of two bytes of `w`, each over two bytes: SIGNS is a selector of PRMT, whose nibbles of 8 and
// more give a byte's sign eight times.
template <uint32_t SIGNS>
__device__ __forceinline__ uint32_t signs(uint32_t w)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(SIGNS));
    return r;
}

// A vector's entries, those not allowed set to -inf.
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 v, uint32_t m)
{
    if (sizeof(T) == 4) {
        return make_uint4(m & 1u ? v.x : 0xFF800000u, m & 2u ? v.y : 0xFF800000u, m & 4u ? v.z : 0xFF800000u,
                          m & 8u ? v.w : 0xFF800000u);
    }
    // each of four bits to the sign of a byte, then each sign over the bytes of its entry
    const uint32_t lo = (m & 15u) * 0x10204080u, hi = (m >> 4) * 0x10204080u;
    const uint32_t k0 = signs<0x9988>(lo), k1 = signs<0xBBAA>(lo), k2 = signs<0x9988>(hi), k3 = signs<0xBBAA>(hi);
    return make_uint4((v.x & k0) | (0xFF80FF80u & ~k0), (v.y & k1) | (0xFF80FF80u & ~k1), (v.z & k2) | (0xFF80FF80u & ~k2),
                      (v.w & k3) | (0xFF80FF80u & ~k3));
}

// ---- asynchronous copies to shared memory --------------------------------------
__device__ __forceinline__ void copy16(void* dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// wait until at most `left` of this thread's last groups are under way
template <int left>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
}

// T: uint16_t for bf16 rows, uint32_t for fp32 rows.  COPY: out of place, by tiles; every row of the two
// matrices starts alike within 16 bytes.
template <typename T, bool COPY>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const __grid_constant__ AdjustArgs a, const AdjustGeom g)
{
    constexpr int kPer = 16 / sizeof(T);            // entries of a vector
    constexpr int kRegion = kAdjTile / sizeof(T);   // ids of a region
    constexpr uint32_t kAll = (1u << kPer) - 1;
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ int32_t s_listed[kAdjWarps];
    const sv_logit_rules& u = a.rules;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t ids = g.slice + kAdjEdge, V = a.in.width;
    const bool biased = g.bias_bits != 0;
    const AdjustLayout at = layout_of(g, COPY);
    uint32_t* s_tab = s_mem + at.tab;
    uint32_t* s_bias = s_mem + at.bias;  // an id's last bias: 1 + its number, 0 for none
    int2* s_row = reinterpret_cast<int2*>(s_mem + at.row);  // each row's mask (-1: none), and the drafts before its branch's
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

    for (int j = tid; j < rows; j += kAdjThreads) {
        int64_t i = -1;
        if (u.mask != nullptr) i = u.mask_row != nullptr ? u.mask_row[first + j] : first + j;
        s_row[j] = make_int2(i >= 0 && i < u.masks ? static_cast<int32_t>(i) : -1,
                             row0 + j > 0 ? (row0 + j - 1) / a.k * a.k : 0);
    }
    // The first tokens are on their way before their number is known: all of the row may be read.
    const int32_t* history = u.history + static_cast<int64_t>(r) * u.history_width;
    const int32_t* draft = a.draft + static_cast<int64_t>(r) * g.drafts;
    int32_t token[kAdjBatch], first_draft = 0, first_bias = 0;
    auto fetch = [&](int32_t (&to)[kAdjBatch], int32_t i0, int32_t end) {
#pragma unroll
        for (int q = 0; q < kAdjBatch; ++q)
            if (i0 + q * kAdjThreads < end) to[q] = history[i0 + q * kAdjThreads];
    };
    if (u.history != nullptr) fetch(token, tid, u.history_width);
    if (tid < g.drafts) first_draft = draft[tid];
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
        if (b0 + tid < b1) first_bias = u.bias_id[b0 + tid];
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
    for (int i = tid; i < (at.row - at.tab) / 4; i += kAdjThreads)
        reinterpret_cast<uint4*>(s_tab)[i] = make_uint4(0, 0, 0, 0);
    if (tid < kAdjWarps) s_listed[tid] = 0;
    __syncthreads();

    // A warp's units: regions of rows, its region the same in each.
    const int32_t units = rows << g.region_shift, region = warp & ((1 << g.region_shift) - 1);
    const int32_t unit0 = warp, in_slice = s0 + region * kRegion;
    struct Row {
        const T* in;
        T* out;
        const uint32_t* mask;  // NULL: none
        int32_t x0;            // id of the region's first entry
        int32_t row;
        int32_t before;        // drafts before those of the row's branch
    };
    auto row_of = [&](int32_t unit) {
        Row w;
        const int32_t j = unit >> g.region_shift;
        w.in = reinterpret_cast<const T*>(a.in.data) + (first + j) * a.in.stride;
        w.out = reinterpret_cast<T*>(const_cast<char*>(a.out.data)) + (first + j) * a.out.stride;
        const int2 i = s_row[j];
        w.mask = i.x < 0 ? nullptr : u.mask + static_cast<int64_t>(i.x) * u.mask_words;
        w.row = row0 + j;
        w.before = i.y;
        w.x0 = in_slice;
        // entries that the row starts behind a 16-byte boundary
        if (COPY || a.in.data == a.out.data)
            w.x0 -= (static_cast<int32_t>(reinterpret_cast<uintptr_t>(w.in)) & 15) / static_cast<int32_t>(sizeof(T));
        return w;
    };
    T* tiles = reinterpret_cast<T*>(s_mem) + warp * kAdjStages * kRegion;
    uint32_t* masks = s_mem + at.mask + warp * kAdjStages * kAdjMaskWords;
    auto bring = [&](int32_t unit, int stage) {
        if (unit < units) {
            const Row w = row_of(unit);
            T* tile = tiles + stage * kRegion;
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) {
                const int32_t o = (q * 32 + lane) * kPer, x = w.x0 + o;
                if (x >= 0 && x + kPer <= V) {
                    copy16(tile + o, w.in + x);
                } else {
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y) tile[y - w.x0] = w.in[y];
                }
            }
            if (w.mask != nullptr) {
                const int32_t word = (w.x0 >> 5) + lane;
                if (word >= 0 && word < u.mask_words) copy4(masks + stage * kAdjMaskWords + lane, w.mask + word);
                if (lane == 0 && word + 32 < u.mask_words && kAdjMaskWords > 32)
                    copy4(masks + stage * kAdjMaskWords + 32, w.mask + word + 32);
            }
        }
        copies_commit();
    };
    if (COPY) {
#pragma unroll
        for (int i = 0; i < kAdjStages - 1; ++i) bring(unit0 + i * kAdjWarps, i);
    }

    // The slice's entry of a token, -1 for none.
    auto meet = [&](int32_t x) -> int32_t {
        if (static_cast<uint32_t>(x) >= static_cast<uint32_t>(V)) {
            st |= SV_ST_TOKEN_RANGE;
            return -1;
        }
        return static_cast<uint32_t>(x - base) < static_cast<uint32_t>(ids) ? x - base : -1;
    };
    for (int32_t i0 = tid; i0 < len; i0 += kAdjThreads * kAdjBatch) {
        int32_t next[kAdjBatch];
        fetch(next, i0 + kAdjThreads * kAdjBatch, len);
#pragma unroll
        for (int q = 0; q < kAdjBatch; ++q) {
            const int32_t i = i0 + q * kAdjThreads;
            const int32_t l = i < len ? meet(token[q]) : -1;
            token[q] = next[q];
            if (l < 0) continue;
            if (i >= prompt)
                atomicAdd(&s_tab[l], 1u);
            else
                atomicOr(&s_tab[l], kAdjSeen);
        }
    }
    for (int32_t i = tid; i < g.drafts; i += kAdjThreads) {
        const int32_t l = meet(i == tid ? first_draft : draft[i]);
        if (l < 0) continue;
        uint32_t old = s_tab[l], was;
        do {
            was = old;
            s_next[i] = static_cast<uint16_t>((was & kAdjHead) >> kAdjHeadShift);
            old = atomicCAS(&s_tab[l], was, (was & ~kAdjHead) | (static_cast<uint32_t>(i + 1) << kAdjHeadShift));
        } while (old != was);
    }
    for (int32_t i = b0 + tid; i < b1; i += kAdjThreads) {
        const int32_t l = meet(i == b0 + tid ? first_bias : u.bias_id[i]);
        if (l < 0) continue;
        const uint32_t entry = static_cast<uint32_t>(i) + 1;
        if (g.bias_bits == 32) {
            atomicMax(&s_bias[l], entry);
        } else {
            uint32_t* word = &s_bias[l >> 1];
            const int half = (l & 1) * 16;
            uint32_t old = *word, was;
            do {
                was = old;
                if (((was >> half) & 0xFFFFu) >= entry) break;
                old = atomicCAS(word, was, (was & ~(0xFFFFu << half)) | (entry << half));
            } while (old != was);
        }
    }
    if (s == 0 && group == 0 && a.status != nullptr) {
        if (u.mask != nullptr && u.mask_row != nullptr)
            for (int32_t i = tid; i < g.rows; i += kAdjThreads)
                if (u.mask_row[static_cast<int64_t>(r) * g.rows + i] >= u.masks) st |= SV_ST_BAD_MASK;
        st |= (__syncthreads_or(st & SV_ST_TOKEN_RANGE) ? SV_ST_TOKEN_RANGE : 0u) |
              (__syncthreads_or(st & SV_ST_BAD_MASK) ? SV_ST_BAD_MASK : 0u);
        if (tid == 0) a.status[r] = static_cast<int32_t>(st);
    }
    __syncthreads();

    // The ids that a rule meets, by regions; the last ones of a region stand in the next one's list, too, for
    // the rows that start within a vector and have them there.
    auto bias_of = [&](int32_t l) -> uint32_t {
        return !biased ? 0u : g.bias_bits == 32 ? s_bias[l] : (s_bias[l >> 1] >> ((l & 1) * 16)) & 0xFFFFu;
    };
    for (int32_t l0 = 4 * tid; l0 < ids; l0 += 4 * kAdjThreads) {
        const uint4 four = *reinterpret_cast<const uint4*>(s_tab + l0);
        uint32_t met = (four.x != 0) | (four.y != 0) << 1 | (four.z != 0) << 2 | (four.w != 0) << 3;
        if (biased)
            for (int e = 0; e < 4; ++e) met |= (bias_of(l0 + e) != 0) << e;
        for (; met != 0; met &= met - 1) {
            const int32_t l = l0 + __ffs(met) - 1, i = l - kAdjEdge, q = i / kRegion;  // 0 for those before the slice, too
            s_list[q * (kRegion + kAdjEdge) + atomicAdd(&s_listed[q], 1)] = static_cast<uint16_t>(l);
            if (i >= 0 && (i + kAdjEdge) / kRegion > q && i + kAdjEdge < g.slice)
                s_list[(q + 1) * (kRegion + kAdjEdge) + atomicAdd(&s_listed[q + 1], 1)] = static_cast<uint16_t>(l);
        }
    }
    __syncthreads();

    // The adjusted entry of the table's id l in a row.
    auto adjusted = [&](const Row& w, int32_t l, T raw) -> T {
        // the drafts before the row: the first i + 1 of branch b, for row 1 + b * k + i
        const uint32_t word = s_tab[l];
        uint32_t count = word & kAdjCount;
        for (uint32_t e = (word & kAdjHead) >> kAdjHeadShift; e != 0; e = s_next[e - 1])
            count += static_cast<int32_t>(e) > w.before && static_cast<int32_t>(e) <= w.row;
        const uint32_t entry = bias_of(l);
        const bool seen = (word & kAdjSeen) != 0 || count != 0;
        if (!seen && entry == 0) return raw;
        float z = widen<T>(raw);
        if (seen) z = z > 0.0f ? z / rep : z * rep;
        if (count != 0) z -= pres + freq * static_cast<float>(count);
        if (entry != 0) z += u.bias_value[entry - 1];
        return narrow<T>(z);
    };
    const uint16_t* list = s_list + region * (kRegion + kAdjEdge);
    const int32_t listed = s_listed[region];

    if (COPY) {
        int stage = 0;
        for (int32_t unit = unit0; unit < units; unit += kAdjWarps) {
            __syncwarp();  // the tile before is stored
            bring(unit + (kAdjStages - 1) * kAdjWarps, stage == 0 ? kAdjStages - 1 : stage - 1);
            copies_wait<kAdjStages - 1>();
            __syncwarp();
            const Row w = row_of(unit);
            T* tile = tiles + stage * kRegion;
            const uint32_t* words = masks + stage * kAdjMaskWords;
            for (int32_t i = lane; i < listed; i += 32) {
                const int32_t l = list[i], o = base + l - w.x0;
                if (o >= 0 && o < kRegion) tile[o] = adjusted(w, l, tile[o]);
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) {
                const int32_t o = (q * 32 + lane) * kPer, x = w.x0 + o;
                uint4 v = *reinterpret_cast<const uint4*>(tile + o);
                uint32_t m = kAll;
                if (w.mask != nullptr) {
                    const int32_t b = (w.x0 & 31) + o;
                    m = __funnelshift_r(words[b >> 5], words[min((b >> 5) + 1, kAdjMaskWords - 1)], b & 31) & kAll;
                    v = masked<T>(v, m);
                }
                if (x >= 0 && x + kPer <= V) {
                    *reinterpret_cast<uint4*>(w.out + x) = v;
                } else {
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y)
                        w.out[y] = (m >> (y - x)) & 1u ? tile[y - w.x0] : kNegInf<T>;
                }
            }
            stage = stage + 1 == kAdjStages ? 0 : stage + 1;
        }
        copies_wait<0>();
        return;
    }

    const bool in_place = a.in.data == a.out.data;
    for (int32_t unit = unit0; unit < units; unit += kAdjWarps) {
        const Row w = row_of(unit);
        if (in_place && w.mask != nullptr) {
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) {
                const int32_t x = w.x0 + (q * 32 + lane) * kPer;
                if (x >= 0 && x + kPer <= V) {
                    const uint32_t lo = w.mask[x >> 5], hi = (x & 31) + kPer > 32 ? w.mask[(x >> 5) + 1] : 0u;
                    const uint32_t m = __funnelshift_r(lo, hi, x & 31) & kAll;
                    uint4* p = reinterpret_cast<uint4*>(w.out + x);
                    if (m != kAll) *p = masked<T>(m != 0u ? *p : make_uint4(0, 0, 0, 0), m);
                } else {
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y)
                        if (!allowed(w.mask, y)) w.out[y] = kNegInf<T>;
                }
            }
        } else if (!in_place) {  // rows that start differently
#pragma unroll 8
            for (int32_t x = w.x0 + lane; x < min(w.x0 + kRegion, V); x += 32)
                w.out[x] = allowed(w.mask, x) ? w.in[x] : kNegInf<T>;
        }
        __syncwarp();
        for (int32_t i = lane; i < listed; i += 32) {
            const int32_t l = list[i], x = base + l;
            if (x >= w.x0 && x < w.x0 + kRegion && allowed(w.mask, x)) w.out[x] = adjusted(w, l, w.in[x]);
        }
    }
}

// Whether the rows of the two matrices start alike within 16 bytes, and are not the same ones.
bool by_tiles(const AdjustArgs& a)
{
    return a.in.data != a.out.data && reinterpret_cast<uintptr_t>(a.in.data) % 16 == reinterpret_cast<uintptr_t>(a.out.data) % 16 &&
           (a.in.stride - a.out.stride) * a.in.esize % 16 == 0;
}

AdjustGeom geom_of(const AdjustArgs& a)
{
    const int sms = std::max(1, device_sm_count());
    AdjustGeom g{};
    g.drafts = a.branches * a.k;
    g.rows = 1 + g.drafts;
    g.bias_bits = a.rules.bias_entries == 0 ? 0 : a.rules.bias_entries <= 0xFFFF ? 16 : 32;
    const int32_t region = kAdjTile / a.in.esize;
    auto slices = [&](int64_t n) { return (static_cast<int64_t>(a.in.width) + kAdjEdge - 1 + n - 1) / n; };
    g.slice = kAdjSlice;
    while (g.slice > region && a.R * slices(g.slice) < 4 * sms) g.slice /= 2;
    while ((region << g.region_shift) < g.slice) ++g.region_shift;
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
    const bool tiles = by_tiles(a), bf16 = a.in.dtype == SV_BF16;
    const int bytes = layout_of(g, tiles).bytes;
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.R) * g.slices * g.groups);
    auto* kernel = tiles ? bf16 ? adjust_kernel<uint16_t, true> : adjust_kernel<uint32_t, true>
                         : bf16 ? adjust_kernel<uint16_t, false> : adjust_kernel<uint32_t, false>;
    if (cudaError_t e = allow_shared(kernel, bytes)) return e;
    kernel<<<blocks, kAdjThreads, bytes, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
