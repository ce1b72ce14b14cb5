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
//
// Bound by bytes less than by what stands before them: 67 us for 576 rows of 151,936 bf16 logits (359 MB, 5.4 TB/s,
// 0.79 of a copy's rate) with 500 to 8,000 tokens a request, 16 biases and masks on two rows of three, of which 55 are
// the copy alone, 2 the scan of every request's tokens in each of its 38 slices, 5 the listed entries, 3 biases and
// drafts, 2 the masks; 33 us for 561 rows of 32,003 fp32 logits (146 MB, 4.4 TB/s).  In place 64 and 27 us, and 41 and
// 18 without masks.  One row of 151,936 takes 4.4 us: a launch, the tokens, a tile.  24 warps share an SM there, so an
// instruction costs a warp about ten cycles, and those that stand before the rows count most.
// A tile in shared memory costs less than computing over the copies afterwards (93 and 41 us at the time), two tiles a
// warp less than three (81 against 103: the third costs a thread block per SM), slices of 4,096 ids less than 8,192 or
// 2,048 (86 and 109 against 80), a thread block an item less than resident ones that walk through items (72 against 88:
// their shares are uneven).  Many tokens of one slice make its block the last one: 94 us where a request's 1,600 ids lie
// side by side.
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
constexpr int kAdjStages = 2;                    // tiles of a warp's ring: one on its way, one in hand
constexpr int kAdjSlice = 4096;                  // most ids of a slice
constexpr int kAdjFewSlice = 8192, kAdjFewRows = 2;  // of one with few rows behind it, and how many those are
constexpr int kAdjEdge = 8;                      // ids before a slice that a row which starts within a vector needs
constexpr int kAdjTokens = 16;                   // tokens of a thread that are brought at a time
constexpr int kAdjMaskWords = kAdjTile / 2 / 32 + 1;  // words of a region's mask

// a word of the table: bit 31 seen, bits 19 .. 30 the head of the chain (0: none), bits 0 .. 18 the count
constexpr uint32_t kAdjSeen = 1u << 31, kAdjHeadShift = 19, kAdjHead = 0xFFFu << kAdjHeadShift,
                   kAdjCount = (1u << kAdjHeadShift) - 1;
static_assert(SV_MAX_HISTORY <= (1 << kAdjHeadShift) - 1, "a count must not reach the chain's head");
static_assert(SV_MAX_BRANCHES * SV_MAX_K < (1 << 12), "a draft's number must fit the head");
static_assert(kAdjSlice / (kAdjTile / 4) <= kAdjWarps && kAdjFewSlice / (kAdjTile / 2) <= kAdjWarps,
              "a warp keeps to one region, and a region has a warp");
static_assert(kAdjFewSlice <= kAdjThreads * 32, "a thread lists 32 ids");
static_assert(kAdjTokens == 16, "a thread reads its tokens four at a time, and 16 bits say which are the slice's");
static_assert(kAdjTokens * 32 * 4 <= kAdjTile, "a warp's tokens wait in a tile");
static_assert(kAdjMaskWords >= 33, "a warp brings 33 words of a mask");

struct AdjustGeom {
    int32_t slice, slices;  // ids of a slice (a power of two), slices of a row
    int32_t region_shift;   // log2 of a slice's regions, at most kAdjWarps
    int32_t rows, groups;   // rows of a request, thread blocks that share them
    int32_t most_rows;      // of a thread block
    int32_t drafts;         // branches * k
    int32_t bias_bits;      // of an id's word in the table of biases: 0 without biases, 16 where their numbers fit, else 32
};

// The parts of a CTA's shared memory, in 32-bit words; the tiles lie first (in place: one a warp, for tokens).
struct AdjustLayout {
    int32_t mask, tab, bias, bits, row, list, next, bytes;  // list and next hold 16 bits each
};
__host__ __device__ inline AdjustLayout layout_of(const AdjustGeom& g, bool tiles)
{
    const int32_t ids = g.slice + kAdjEdge;
    AdjustLayout l;
    l.mask = kAdjWarps * (tiles ? kAdjStages : 1) * kAdjTile / 4;
    l.tab = l.mask + (tiles ? (kAdjWarps * kAdjStages * kAdjMaskWords + 3) / 4 * 4 : 0);
    l.bias = l.tab + ids;
    l.bits = l.bias + ids * g.bias_bits / 32;
    l.row = l.bits + g.slice / 32 + 4;
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
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_kernel(const __grid_constant__ AdjustArgs a, const AdjustGeom g)
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
    uint32_t* s_bits = s_mem + at.bits;  // the slice's ids that a rule meets, then those before it
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

    // A warp takes one region, in every kAdjWarps / regions-th row from row j0 on.
    const int32_t region = warp & ((1 << g.region_shift) - 1), in_slice = s0 + region * kRegion;
    const int32_t j0 = warp >> g.region_shift, j_step = kAdjWarps >> g.region_shift;
    const bool in_place = a.in.data == a.out.data;
    const T* in = reinterpret_cast<const T*>(a.in.data) + (first + j0) * a.in.stride;
    T* out = reinterpret_cast<T*>(const_cast<char*>(a.out.data)) + (first + j0) * a.out.stride;
    const int64_t in_step = j_step * a.in.stride, out_step = j_step * a.out.stride;
    // The id of a row's first entry of the region: rows may start within 16 bytes.
    auto region_of = [&](const T* row) -> int32_t {
        return COPY || in_place ? in_slice - (static_cast<int32_t>(reinterpret_cast<uintptr_t>(row)) & 15) / static_cast<int32_t>(sizeof(T))
                                : in_slice;
    };
    uint8_t* tiles = reinterpret_cast<uint8_t*>(s_mem) + warp * (COPY ? kAdjStages : 1) * kAdjTile;
    uint32_t* masks = s_mem + at.mask + warp * kAdjStages * kAdjMaskWords;
    auto mask_at = [&](int32_t i) -> const uint32_t* {
        return i < 0 ? nullptr : u.mask + static_cast<int64_t>(i) * u.mask_words;
    };
    // a row's region on its way to a tile
    auto bring = [&](const T* row, int stage) {
        const int32_t x0 = region_of(row);
        uint8_t* tile = tiles + stage * kAdjTile;
        if (x0 >= 0 && x0 + kRegion <= V) {
            const uint4* src = reinterpret_cast<const uint4*>(row + x0) + lane;
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) copy16(tile + (q * 32 + lane) * 16, src + q * 32);
        } else {
#pragma unroll 1
            for (int q = 0; q < kAdjVecs; ++q) {
                const int32_t o = (q * 32 + lane) * kPer, x = x0 + o;
                if (x >= 0 && x + kPer <= V) {
                    copy16(tile + o * sizeof(T), row + x);
                } else {
#pragma unroll 1
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y) reinterpret_cast<T*>(tile)[y - x0] = row[y];
                }
            }
        }
    };
    // its mask's words: those of a region that does not begin with a word reach into one more
    auto bring_mask = [&](const T* row, int32_t i, int stage) {
        if (i < 0) return;
        const int32_t x0 = region_of(row), word = (x0 >> 5) + lane;
        const uint32_t* from = mask_at(i) + word;
        uint32_t* to = masks + stage * kAdjMaskWords + lane;
        if (static_cast<uint32_t>(word) < static_cast<uint32_t>(u.mask_words)) copy4(to, from);
        if ((x0 & 31) != 0 && lane == 0 && word + 32 < u.mask_words) copy4(to + 32, from + 32);
    };
    // row j's mask as it was asked for, and as an index (-1: none)
    const bool rows_ask = u.mask != nullptr && u.mask_row != nullptr;
    auto asked_mask = [&](int32_t j) -> int32_t { return rows_ask && j < rows ? u.mask_row[first + j] : 0; };
    auto mask_index = [&](int32_t asked, int32_t j) -> int32_t {
        const int64_t i = rows_ask ? asked : first + j;
        return u.mask != nullptr && i >= 0 && i < u.masks ? static_cast<int32_t>(i) : -1;
    };

    // The first tile and the first tokens are on their way before anything is known of the request: all of a row of
    // the history may be read.  The tokens wait in the tile that comes into use last.
    const int32_t* history = u.history + static_cast<int64_t>(r) * u.history_width;
    int32_t* tokens = reinterpret_cast<int32_t*>(tiles + (COPY ? kAdjStages - 1 : 0) * kAdjTile) + 4 * lane;
    const bool by_four = (reinterpret_cast<uintptr_t>(history) & 15) == 0;
    // Of the tokens i0 .. end - 1 four in 1,024 are this thread's; it alone reads them.
    auto bring_tokens = [&](int32_t i0, int32_t end) {
#pragma unroll
        for (int q = 0; q < kAdjTokens / 4; ++q) {
            const int32_t i = i0 + 4 * (q * kAdjThreads + tid);
            if (by_four && i + 4 <= end) {
                copy16(tokens + q * 128, history + i);
            } else {
#pragma unroll 1
                for (int e = 0; e < 4 && i + e < end; ++e) copy4(tokens + q * 128 + e, history + i + e);
            }
        }
    };
    if (COPY && j0 < rows) bring(in, 0);
    if (u.history != nullptr) bring_tokens(0, u.history_width);
    copies_commit();
    const int32_t* draft = a.draft + static_cast<int64_t>(r) * g.drafts;
    const int32_t first_draft = tid < g.drafts ? draft[tid] : 0;
    const int32_t first_mask = COPY ? asked_mask(j0) : 0, row_mask = asked_mask(tid);
    const int32_t asked_len = u.history != nullptr ? u.history_len[r] : 0;
    const int32_t asked_prompt = u.history != nullptr && u.prompt_len != nullptr ? u.prompt_len[r] : 0;
    const int32_t asked_b0 = biased ? u.bias_start[r] : 0, asked_b1 = biased ? u.bias_start[r + 1] : 0;
    float rep = u.repetition != nullptr ? u.repetition[r] : 1.0f;
    float pres = u.presence != nullptr ? u.presence[r] : 0.0f;
    float freq = u.frequency != nullptr ? u.frequency[r] : 0.0f;
    for (int i = tid; i < (at.row - at.tab) / 4; i += kAdjThreads)
        reinterpret_cast<uint4*>(s_tab)[i] = make_uint4(0, 0, 0, 0);
    if (tid < kAdjWarps) s_listed[tid] = 0;
    for (int j = tid; j < rows; j += kAdjThreads)
        s_row[j] = make_int2(mask_index(j == tid ? row_mask : asked_mask(j), j),
                             row0 + j > 0 ? (row0 + j - 1) / a.k * a.k : 0);
    if (COPY && j0 < rows) bring_mask(in, mask_index(first_mask, j0), 0);
    copies_commit();
    __syncthreads();

    // what cannot be asked for is left out or cut
    uint32_t st = 0;
    const int32_t b0 = min(max(asked_b0, 0), u.bias_entries), b1 = min(max(asked_b1, b0), u.bias_entries);
    const int32_t first_bias = b0 + tid < b1 ? u.bias_id[b0 + tid] : 0;
    const int32_t len = min(max(asked_len, 0), u.history_width), prompt = min(max(asked_prompt, 0), len);
    if (len != asked_len || prompt != asked_prompt || b0 != asked_b0 || b1 != asked_b1) st |= SV_ST_BAD_LENGTH;
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

    // Tokens of the vocabulary that are the slice's: low .. low + span - 1.
    const bool tells = s == 0 && group == 0 && a.status != nullptr;
    const int32_t low = max(base, 0);
    const uint32_t span = static_cast<uint32_t>(max(min(base + ids, V) - low, 0));
    bool outside = false;
    auto meets = [&](int32_t x) -> bool {
        if (tells) outside = outside || static_cast<uint32_t>(x) >= static_cast<uint32_t>(V);
        return static_cast<uint32_t>(x - low) < span;
    };
    // Notes that a rule meets an id, and gives the id's place in the table.
    auto place = [&](int32_t x) -> int32_t {
        const int32_t i = x - s0;
        atomicOr(i >= 0 ? &s_bits[i >> 5] : &s_bits[g.slice / 32], 1u << (i >= 0 ? i & 31 : i + kAdjEdge));
        return x - base;
    };
    copies_wait<1>();  // the tokens
    for (int32_t i0 = 0; i0 < len;) {
        uint32_t hits = 0, wrong = 0;  // which of this thread's tokens are the slice's (most have none), or nobody's
#pragma unroll
        for (int q = 0; q < kAdjTokens / 4; ++q) {
            if (i0 + 4 * q * kAdjThreads >= len) break;
            const int4 x = *reinterpret_cast<const int4*>(tokens + q * 128);
            const uint32_t brought = (1u << min(max(len - (i0 + 4 * (q * kAdjThreads + tid)), 0), 4)) - 1;
            auto below = [&](int32_t from, uint32_t n) -> uint32_t {  // which are from .. from + n - 1
                return (static_cast<uint32_t>(x.x - from) < n) | (static_cast<uint32_t>(x.y - from) < n) << 1 |
                       (static_cast<uint32_t>(x.z - from) < n) << 2 | (static_cast<uint32_t>(x.w - from) < n) << 3;
            };
            hits |= (below(low, span) & brought) << (4 * q);
            if (tells) wrong |= ~below(0, static_cast<uint32_t>(V)) & brought;
        }
        outside = outside || wrong != 0;
        for (; hits != 0; hits &= hits - 1) {
            const int q = __ffs(hits) - 1;
            const int32_t l = place(tokens[q / 4 * 128 + q % 4]);
            if (i0 + 4 * (q / 4 * kAdjThreads + tid) + q % 4 >= prompt)
                atomicAdd(&s_tab[l], 1u);
            else
                atomicOr(&s_tab[l], kAdjSeen);
        }
        i0 += kAdjThreads * kAdjTokens;
        if (i0 < len) {
            bring_tokens(i0, len);
            copies_commit();
            copies_wait<0>();
        }
    }
    for (int32_t i = tid; i < g.drafts; i += kAdjThreads) {
        const int32_t x = i == tid ? first_draft : draft[i];
        if (!meets(x)) continue;
        uint32_t* word = &s_tab[place(x)];
        uint32_t old = *word, was;
        do {
            was = old;
            s_next[i] = static_cast<uint16_t>((was & kAdjHead) >> kAdjHeadShift);
            old = atomicCAS(word, was, (was & ~kAdjHead) | (static_cast<uint32_t>(i + 1) << kAdjHeadShift));
        } while (old != was);
    }
    for (int32_t i = b0 + tid; i < b1; i += kAdjThreads) {
        const int32_t x = i == b0 + tid ? first_bias : u.bias_id[i];
        if (!meets(x)) continue;
        const int32_t l = place(x);
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
    if (tells) {
        bool over = false;
        if (u.mask != nullptr && u.mask_row != nullptr)
            for (int32_t i = tid; i < g.rows; i += kAdjThreads)
                over = over || u.mask_row[static_cast<int64_t>(r) * g.rows + i] >= u.masks;
        if (__syncthreads_or(outside)) st |= SV_ST_TOKEN_RANGE;
        if (__syncthreads_or(over)) st |= SV_ST_BAD_MASK;
        if (tid == 0) a.status[r] = static_cast<int32_t>(st);
    }
    __syncthreads();

    // The ids that a rule meets, by regions.  The last ones before a region stand in its list, too, for the rows that
    // start within a vector and have them there.
    auto bias_of = [&](int32_t l) -> uint32_t {
        return !biased ? 0u : g.bias_bits == 32 ? s_bias[l] : (s_bias[l >> 1] >> ((l & 1) * 16)) & 0xFFFFu;
    };
    auto note = [&](int32_t p, int32_t l0, uint32_t met) {
        if (met == 0) return;
        uint16_t* to = s_list + p * (kRegion + kAdjEdge) + atomicAdd(&s_listed[p], __popc(met));
        for (; met != 0; met &= met - 1) *to++ = static_cast<uint16_t>(l0 + __ffs(met) - 1);
    };
    if (32 * tid < g.slice) {
        const uint32_t met = s_bits[tid];
        note(32 * tid / kRegion, kAdjEdge + 32 * tid, met);
        const int32_t after = (32 * tid + 32) / kRegion;  // the region that begins behind these ids
        if ((32 * tid + 32) % kRegion == 0 && after < 1 << g.region_shift)
            note(after, kAdjEdge + 32 * tid + 24, met >> 24);
    }
    if (tid == 0) note(0, 0, s_bits[g.slice / 32]);
    __syncthreads();

    // The adjusted entry of the table's id l in row j.
    auto adjusted = [&](int32_t j, int32_t l, T raw) -> T {
        // the drafts before the row: the first i + 1 of branch b, for row 1 + b * k + i
        const uint32_t word = s_tab[l];
        uint32_t count = word & kAdjCount;
        for (uint32_t e = (word & kAdjHead) >> kAdjHeadShift; e != 0; e = s_next[e - 1])
            count += static_cast<int32_t>(e) > s_row[j].y && static_cast<int32_t>(e) <= row0 + j;
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
        for (int32_t j = j0; j < rows; j += j_step, out += out_step) {
            __syncwarp();  // the tile before is stored
            in += in_step;
            if (j + j_step < rows) {
                bring(in, stage ^ 1);
                bring_mask(in, s_row[j + j_step].x, stage ^ 1);
            }
            copies_commit();
            copies_wait<1>();
            __syncwarp();
            const int32_t x0 = region_of(out);
            T* tile = reinterpret_cast<T*>(tiles + stage * kAdjTile);
            const uint32_t* words = masks + stage * kAdjMaskWords;
            for (int32_t i = lane; i < listed; i += 32) {
                const int32_t l = list[i], o = base + l - x0;
                if (static_cast<uint32_t>(o) < static_cast<uint32_t>(kRegion)) tile[o] = adjusted(j, l, tile[o]);
            }
            __syncwarp();
            const bool has_mask = s_row[j].x >= 0;
            auto bits_of = [&](int32_t o) -> uint32_t {
                const int32_t b = (x0 & 31) + o;
                return __funnelshift_r(words[b >> 5], words[min((b >> 5) + 1, kAdjMaskWords - 1)], b & 31) & kAll;
            };
            const uint4* from = reinterpret_cast<const uint4*>(tile) + lane;
            if (x0 >= 0 && x0 + kRegion <= V) {
                uint4* to = reinterpret_cast<uint4*>(out + x0) + lane;
                if (!has_mask) {
#pragma unroll
                    for (int q = 0; q < kAdjVecs; ++q) to[q * 32] = from[q * 32];
                } else if (x0 % 8 == 0) {  // a vector's bits lie in one byte
                    const uint8_t* bits = reinterpret_cast<const uint8_t*>(words) + ((x0 & 31) + lane * kPer) / 8;
#pragma unroll
                    for (int q = 0; q < kAdjVecs; ++q)
                        to[q * 32] = masked<T>(from[q * 32], kPer == 8 ? bits[q * 4 * kPer] : (bits[q * 4 * kPer] >> (lane * kPer % 8)) & kAll);
                } else {
#pragma unroll
                    for (int q = 0; q < kAdjVecs; ++q) to[q * 32] = masked<T>(from[q * 32], bits_of((q * 32 + lane) * kPer));
                }
            } else {
#pragma unroll 1
                for (int q = 0; q < kAdjVecs; ++q) {
                    const int32_t o = (q * 32 + lane) * kPer, x = x0 + o;
                    const uint32_t m = has_mask ? bits_of(o) : kAll;
                    if (x >= 0 && x + kPer <= V) {
                        *reinterpret_cast<uint4*>(out + x) = masked<T>(from[q * 32], m);
                    } else {
#pragma unroll 1
                        for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y)
                            out[y] = (m >> (y - x)) & 1u ? tile[y - x0] : kNegInf<T>;
                    }
                }
            }
            stage ^= 1;
        }
        copies_wait<0>();
        return;
    }

    if (!in_place) {  // rows that start differently
        for (int32_t j = j0; j < rows; j += j_step, in += in_step, out += out_step) {
            const uint32_t* mask = mask_at(s_row[j].x);
#pragma unroll 8
            for (int32_t x = in_slice + lane; x < min(in_slice + kRegion, V); x += 32)
                out[x] = allowed(mask, x) ? in[x] : kNegInf<T>;
            __syncwarp();
            for (int32_t i = lane; i < listed; i += 32) {
                const int32_t l = list[i], x = base + l;
                if (x >= in_slice && x < in_slice + kRegion && allowed(mask, x)) out[x] = adjusted(j, l, in[x]);
            }
        }
        return;
    }

    // In place: a lane has 32 ids' bits of the row's mask, brought while the row before was written, and the
    // first listed entries are read while the masked ones are written.
    uint32_t lo = 0, hi = 0;
    auto read_mask = [&](const T* row, int32_t j) {
        lo = hi = 0xFFFFFFFFu;
        const uint32_t* mask = j < rows ? mask_at(s_row[j].x) : nullptr;
        if (mask == nullptr) return;
        const int32_t word = (region_of(row) >> 5) + lane;
        if (word >= 0 && word < u.mask_words) lo = mask[word];
        if (word + 1 < u.mask_words) hi = mask[word + 1];
    };
    read_mask(out, j0);
    for (int32_t j = j0; j < rows; j += j_step, out += out_step) {
        const int32_t x0 = region_of(out);
        const bool has_mask = s_row[j].x >= 0;
        const uint32_t bits = __funnelshift_r(lo, hi, x0 & 31);  // of ids x0 + 32 * lane on
        read_mask(out + out_step, j + j_step);
        auto entry = [&](int32_t i, int32_t& l) -> int32_t {  // listed id i's place in the region, -1 for none
            l = i < listed ? list[i] : 0;
            const int32_t o = base + l - x0;
            const bool here = i < listed && static_cast<uint32_t>(o) < static_cast<uint32_t>(kRegion);
            const uint32_t word = __shfl_sync(0xFFFFFFFFu, bits, (o >> 5) & 31);
            return here && ((word >> (o & 31)) & 1u) ? o : -1;
        };
        int32_t l;
        const int32_t o = entry(lane, l);
        T raw = 0;
        if (o >= 0) raw = out[x0 + o];
        if (has_mask) {
            uint32_t m[kAdjVecs];
            uint4 v[kAdjVecs];
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) {
                const int word = q * kPer;  // of the warp's, plus lane * kPer / 32
                m[q] = (__shfl_sync(0xFFFFFFFFu, bits, word + lane * kPer / 32) >> (lane * kPer % 32)) & kAll;
                const int32_t x = x0 + (q * 32 + lane) * kPer;
                // what is masked need not be read
                if (x >= 0 && x + kPer <= V && m[q] != 0u && m[q] != kAll) v[q] = *reinterpret_cast<const uint4*>(out + x);
            }
#pragma unroll
            for (int q = 0; q < kAdjVecs; ++q) {
                const int32_t x = x0 + (q * 32 + lane) * kPer;
                if (x >= 0 && x + kPer <= V) {
                    if (m[q] != kAll) *reinterpret_cast<uint4*>(out + x) = masked<T>(v[q], m[q]);
                } else {
#pragma unroll 1
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y)
                        if (!((m[q] >> (y - x)) & 1u)) out[y] = kNegInf<T>;
                }
            }
            __syncwarp();
        }
        if (o >= 0) out[x0 + o] = adjusted(j, l, raw);
        for (int32_t i = 32; i < listed; i += 32) {
            const int32_t p = entry(i + lane, l);
            if (p >= 0) out[x0 + p] = adjusted(j, l, out[x0 + p]);
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
    // a row or two are little work behind a table, and the request's tokens are looked through for every slice: 256 rows
    // of 256 requests take 88 us with slices of 8,192 bf16 entries and 103 with 4,096; four rows each 36 and 39
    g.slice = g.rows <= kAdjFewRows ? std::min(kAdjFewSlice, kAdjWarps * region) : kAdjSlice;
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
