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
// drafts, 2 the masks; 33 us for 561 rows of 32,003 fp32 logits (146 MB, 4.4 TB/s).  In place 66 and 36 us, and 48 and
// 20 without masks.  Rows of the two matrices that start differently within 16 bytes go entry by entry: 576 rows of 151,935
// whose output has no room between its rows take 303 us, and 71 where both have the same.  One row of 151,936 takes 4.4 us: a launch, the tokens, a tile.  24 warps share an SM there, so an
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
constexpr int kAdjEdge = 8;                      // ids before a slice that a row which starts within a vector needs
constexpr int kAdjTokens = 16;                   // tokens of a thread that are brought at a time
constexpr int kAdjMaskWords = kAdjTile / 2 / 32 + 1;  // words of a region's mask

// a word of the table: bit 31 seen, bits 19 .. 30 the head of the chain (0: none), bits 0 .. 18 the count
constexpr uint32_t kAdjSeen = 1u << 31, kAdjHeadShift = 19, kAdjHead = 0xFFFu << kAdjHeadShift,
                   kAdjCount = (1u << kAdjHeadShift) - 1;
static_assert(SV_MAX_HISTORY <= (1 << kAdjHeadShift) - 1, "a count must not reach the chain's head");
static_assert(SV_MAX_BRANCHES * SV_MAX_K < (1 << 12), "a draft's number must fit the head");
static_assert(kAdjSlice / (kAdjTile / 4) <= kAdjWarps, "a warp keeps to one region, and a region has a warp");
static_assert(kAdjSlice <= kAdjThreads * 32, "a thread lists 32 ids");
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

// What a request asks for, and what of it is done: what cannot be asked for is left out or cut.
struct Rules {
    int32_t len, prompt, b0, b1;
    float rep, pres, freq;
};
__device__ __forceinline__ Rules asked_of(const AdjustArgs& a, int32_t r)
{
    const sv_logit_rules& u = a.rules;
    Rules q;
    q.len = u.history != nullptr ? u.history_len[r] : 0;
    q.prompt = u.history != nullptr && u.prompt_len != nullptr ? u.prompt_len[r] : 0;
    q.b0 = u.bias_entries != 0 ? u.bias_start[r] : 0;
    q.b1 = u.bias_entries != 0 ? u.bias_start[r + 1] : 0;
    q.rep = u.repetition != nullptr ? u.repetition[r] : 1.0f;
    q.pres = u.presence != nullptr ? u.presence[r] : 0.0f;
    q.freq = u.frequency != nullptr ? u.frequency[r] : 0.0f;
    return q;
}
__device__ __forceinline__ Rules rules_of(const AdjustArgs& a, const Rules& q, uint32_t& st)
{
    const sv_logit_rules& u = a.rules;
    Rules o;
    o.b0 = min(max(q.b0, 0), u.bias_entries);
    o.b1 = min(max(q.b1, o.b0), u.bias_entries);
    o.len = min(max(q.len, 0), u.history_width);
    o.prompt = min(max(q.prompt, 0), o.len);
    if (o.len != q.len || o.prompt != q.prompt || o.b0 != q.b0 || o.b1 != q.b1) st |= SV_ST_BAD_LENGTH;
    const bool rep_ok = q.rep > 0.0f && !isinf(q.rep), pres_ok = isfinite(q.pres), freq_ok = isfinite(q.freq);
    o.rep = rep_ok ? q.rep : 1.0f;
    o.pres = pres_ok ? q.pres : 0.0f;
    o.freq = freq_ok ? q.freq : 0.0f;
    if (!rep_ok || !pres_ok || !freq_ok) st |= SV_ST_BAD_PENALTY;
    return o;
}

// An entry whose id stands `count` times in the output and, if `seen`, in the prompt; `bias` may be null.
template <typename T>
__device__ __forceinline__ T adjust(T raw, bool seen, uint32_t count, const float* bias, const Rules& ru)
{
    seen = seen || count != 0;
    if (!seen && bias == nullptr) return raw;
    float z = widen<T>(raw);
    if (seen) z = z > 0.0f ? z / ru.rep : z * ru.rep;
    if (count != 0) z -= ru.pres + ru.freq * static_cast<float>(count);
    if (bias != nullptr) z += *bias;
    return narrow<T>(z);
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
    const Rules asked = asked_of(a, r);
    for (int i = tid; i < (at.row - at.tab) / 4; i += kAdjThreads)
        reinterpret_cast<uint4*>(s_tab)[i] = make_uint4(0, 0, 0, 0);
    if (tid < kAdjWarps) s_listed[tid] = 0;
    for (int j = tid; j < rows; j += kAdjThreads)
        s_row[j] = make_int2(mask_index(j == tid ? row_mask : asked_mask(j), j),
                             row0 + j > 0 ? (row0 + j - 1) / a.k * a.k : 0);
    if (COPY && j0 < rows) bring_mask(in, mask_index(first_mask, j0), 0);
    copies_commit();
    __syncthreads();

    uint32_t st = 0;
    const Rules ru = rules_of(a, asked, st);
    const int32_t b0 = ru.b0, b1 = ru.b1, len = ru.len, prompt = ru.prompt;
    const int32_t first_bias = b0 + tid < b1 ? u.bias_id[b0 + tid] : 0;

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
        return adjust<T>(raw, (word & kAdjSeen) != 0, count, entry != 0 ? &u.bias_value[entry - 1] : nullptr, ru);
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

// ---- requests of few rows -------------------------------------------------------
// A table that has a word for every id of a slice costs more than a row or two behind it.  Here a thread block takes a
// long slice, and its table has words only for the ids that a rule meets: they are marked in a bit map first, and an
// id's place is the number of marks before it, from the marks before its word and those of its word.  Then the tokens
// are counted, the rows are copied and masked, and the marked entries are written once more from what they were.  Where
// more ids are marked than the table has words, they are taken in windows, with the tokens gone through for each.
//
// 256 requests of one row of 151,936 bf16 logits with 500 to 8,000 tokens take 44 us so, 37 in place and 22 without
// masks, and 103, 95 and 81 with a word for every id (the copy's bytes alone: 24); 512 of them with up to 2,000 tokens 71, 53
// and 26, and 160, 151 and 122.  A call of up to 100 tokens a
// request takes 35, 22 and 9.  What is left: 256 blocks do not fill 152 SMs evenly, and a block's steps wait for one
// another.  512 threads, two blocks an SM, each with as much of a row as lets all
// blocks be resident at once: with 1,024 and one block 47, 256 and four 65, three blocks an SM 54, slices of which four
// times as many blocks would be resident 57.  Entries met and tokens brought two or four at a time spill or save nothing
// (43 and 46).
// Every window of 4,096 marks goes through all of a request's tokens once more, so long histories cost most where ids
// hardly repeat: 256 requests of 32,000 such tokens take 230 us (the other kernel: 443), of 100,000 1,220 (1,357), and with
// ids by a power of their rank 150 and 686 (377 and 1,097).  The other kernel spreads a request over 38 blocks, so it is the
// faster one where a few requests of many are far longer than the rest, which the host does not know: 4 of 256 with 100,000
// tokens take 852 us here and 136 there, with 500,000 5,800 and 374.  Shorter slices wherever histories may be long (32,768
// ids: 218 and 1,450) cost batches of even lengths: 64 of 100,000 tokens 365 us for 262.
constexpr int kFewThreads = 512;
constexpr int kFewBlocks = 2;      // an SM
constexpr int kFewSlice = 262144;  // most ids of a slice, and the least where there are few
constexpr int kFewLeast = 8192;
constexpr int kFewTable = 4096;    // most words of a table
constexpr int kFewVecs = 4;        // vectors of a row that a thread moves at a time
// Most rows of a request, out of place and in place: 256 requests of three rows take 107 us so and 119 with the other
// kernel (205 of three whose ids hardly repeat 134 and 107), 64 of four 48 and 41; in place 64 of four 35 and 41, of eight
// 55 and 58, and 64 of 33 rows of 32,000 79 and 53.
constexpr int kFewRows = 3, kFewRowsInPlace = 8;

struct FewGeom {
    int32_t slice, slices;
    int32_t rows, drafts;
    int32_t table;  // words
};

struct FewLayout {
    int32_t tab, bias, rank, list, next, row, bytes;  // next holds 16 bits each; the bits lie first
};
__host__ __device__ inline FewLayout few_layout(const FewGeom& g, bool biased)
{
    const int32_t words = g.slice / 32 + 1;
    FewLayout l;
    l.tab = (words + 3) / 4 * 4;
    l.bias = l.tab + g.table;
    l.rank = l.bias + (biased ? g.table : 0);
    l.list = l.rank + words;
    l.next = l.list + g.table;
    l.row = l.next + (g.drafts + 1) / 2;
    l.bytes = 4 * (l.row + g.rows);
    return l;
}

enum class Lie { InPlace, Alike, Apart };  // Apart: they start differently within 16 bytes

template <typename T, Lie HOW>
__global__ void __launch_bounds__(kFewThreads, kFewBlocks) adjust_few_kernel(const __grid_constant__ AdjustArgs a, const FewGeom g)
{
    constexpr int kPer = 16 / sizeof(T);
    constexpr uint32_t kAll = (1u << kPer) - 1;
    extern __shared__ __align__(16) uint32_t s_mem[];
    __shared__ int32_t s_warp[kFewThreads / 32];
    const sv_logit_rules& u = a.rules;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t V = a.in.width, words = g.slice / 32 + 1;
    const bool biased = u.bias_entries != 0;
    const FewLayout at = few_layout(g, biased);
    uint32_t* s_bits = s_mem;
    uint32_t* s_tab = s_mem + at.tab;
    uint32_t* s_bias = s_mem + at.bias;
    int32_t* s_rank = reinterpret_cast<int32_t*>(s_mem + at.rank);
    int32_t* s_list = reinterpret_cast<int32_t*>(s_mem + at.list);
    uint16_t* s_next = reinterpret_cast<uint16_t*>(s_mem + at.next);
    int32_t* s_row = reinterpret_cast<int32_t*>(s_mem + at.row);  // each row's mask, -1 for none

    const int32_t s = static_cast<int32_t>(blockIdx.x % g.slices), r = static_cast<int32_t>(blockIdx.x / g.slices);
    const int32_t s0 = s * g.slice, base = s0 - 32;  // id of the first bit
    const int64_t first = static_cast<int64_t>(r) * g.rows;
    const T* in = reinterpret_cast<const T*>(a.in.data) + first * a.in.stride;
    T* out = reinterpret_cast<T*>(const_cast<char*>(a.out.data)) + first * a.out.stride;
    // The id of a row's first entry of the slice: rows may start within 16 bytes.
    auto start_of = [&](const T* row) -> int32_t {
        return HOW == Lie::Apart ? s0 : s0 - (static_cast<int32_t>(reinterpret_cast<uintptr_t>(row)) & 15) / static_cast<int32_t>(sizeof(T));
    };
    auto mask_at = [&](int32_t i) -> const uint32_t* {
        return i < 0 ? nullptr : u.mask + static_cast<int64_t>(i) * u.mask_words;
    };
    const int32_t* history = u.history + static_cast<int64_t>(r) * u.history_width;
    const bool by_four = (reinterpret_cast<uintptr_t>(history) & 15) == 0;
    const int32_t* draft = a.draft + static_cast<int64_t>(r) * g.drafts;
    const Rules asked = asked_of(a, r);
    for (int32_t i = tid; i < words; i += kFewThreads) s_bits[i] = 0;
    bool over = false;
    for (int32_t j = tid; j < g.rows; j += kFewThreads) {
        const int64_t i = u.mask == nullptr ? -1 : u.mask_row != nullptr ? u.mask_row[first + j] : first + j;
        over = over || (u.mask != nullptr && u.mask_row != nullptr && i >= u.masks);
        s_row[j] = i >= 0 && i < u.masks ? static_cast<int32_t>(i) : -1;
    }
    __syncthreads();

    // The rows, masked.
    auto stream = [&]() {
        for (int32_t j = 0; j < g.rows; ++j) {
            const T* src = in + j * a.in.stride;
            T* dst = out + j * a.out.stride;
            const uint32_t* mask = mask_at(s_row[j]);
            if (HOW == Lie::InPlace && mask == nullptr) continue;
            if (HOW == Lie::Apart) {
#pragma unroll 8
                for (int32_t x = s0 + tid; x < min(s0 + g.slice, V); x += kFewThreads)
                    dst[x] = allowed(mask, x) ? src[x] : kNegInf<T>;
                continue;
            }
            // a warp's vectors lie side by side, and each lane has 32 of their ids' bits
            constexpr int kSpan = kFewVecs * 32 * kPer;
            for (int32_t n = warp * kSpan; n < g.slice; n += kFewThreads / 32 * kSpan) {
                const int32_t x0 = start_of(dst) + n;
                const bool inside = x0 >= 0 && x0 + kSpan <= V;
                uint4 v[kFewVecs];
                uint32_t m[kFewVecs];
                const T* from = src + x0 + lane * kPer;
                T* to = dst + x0 + lane * kPer;
                if (HOW == Lie::Alike && inside) {
#pragma unroll
                    for (int q = 0; q < kFewVecs; ++q) v[q] = *reinterpret_cast<const uint4*>(from + q * 32 * kPer);
                }
                uint32_t bits = 0xFFFFFFFFu;
                if (mask != nullptr) {
                    const int32_t word = (x0 >> 5) + lane;
                    uint32_t lo = 0, hi = 0;
                    if (word >= 0 && word < u.mask_words) lo = mask[word];
                    if ((x0 & 31) != 0 && word + 1 < u.mask_words) hi = mask[word + 1];
                    bits = __funnelshift_r(lo, hi, x0 & 31);
                }
#pragma unroll
                for (int q = 0; q < kFewVecs; ++q)
                    m[q] = (__shfl_sync(0xFFFFFFFFu, bits, q * kPer + lane * kPer / 32) >> (lane * kPer % 32)) & kAll;
                if (inside) {
                    if (HOW == Lie::InPlace) {  // what is masked or stays need not be read
#pragma unroll
                        for (int q = 0; q < kFewVecs; ++q)
                            if (m[q] != 0u && m[q] != kAll) v[q] = *reinterpret_cast<const uint4*>(from + q * 32 * kPer);
                    }
#pragma unroll
                    for (int q = 0; q < kFewVecs; ++q)
                        if (HOW == Lie::Alike || m[q] != kAll) *reinterpret_cast<uint4*>(to + q * 32 * kPer) = masked<T>(v[q], m[q]);
                    continue;
                }
#pragma unroll
                for (int q = 0; q < kFewVecs; ++q) {
                    const int32_t x = x0 + (q * 32 + lane) * kPer;
#pragma unroll 1
                    for (int32_t y = max(x, 0); y < min(x + kPer, V); ++y) {
                        if (!((m[q] >> (y - x)) & 1u))
                            dst[y] = kNegInf<T>;
                        else if (HOW == Lie::Alike)
                            dst[y] = src[y];
                    }
                }
            }
        }
    };
    // Half of the blocks copy first, so that some copy while others count: 256 rows take 42 us so, 44 where all copy first or
    // last.  In place little is copied: 31 and 20 us where all begin with it, 32 and 21 where half do.
    const bool early = HOW == Lie::InPlace || blockIdx.x < gridDim.x / 2;
    if (early) stream();

    uint32_t st = 0;
    const Rules ru = rules_of(a, asked, st);
    const bool tells = s == 0 && a.status != nullptr;
    const int32_t low = max(s0 - kAdjEdge, 0);
    const uint32_t span = static_cast<uint32_t>(max(min(s0 + g.slice, V) - low, 0));
    bool outside = false;
    auto each_token = [&](auto&& f) {
        if (by_four) {
            const int32_t fours = ru.len / 4;
            for (int32_t i = tid; i < fours; i += kFewThreads) {
                const int4 x = reinterpret_cast<const int4*>(history)[i];
                f(4 * i, x.x);
                f(4 * i + 1, x.y);
                f(4 * i + 2, x.z);
                f(4 * i + 3, x.w);
            }
            const int32_t i = 4 * fours + tid;
            if (i < ru.len) f(i, history[i]);
        } else {
            for (int32_t i = tid; i < ru.len; i += kFewThreads) f(i, history[i]);
        }
    };
    auto mark = [&](int32_t x) {
        if (static_cast<uint32_t>(x - low) < span) atomicOr(&s_bits[(x - base) >> 5], 1u << (x & 31));
    };
    each_token([&](int32_t, int32_t x) {
        outside = outside || static_cast<uint32_t>(x) >= static_cast<uint32_t>(V);
        mark(x);
    });
    for (int32_t i = tid; i < g.drafts; i += kFewThreads) {
        const int32_t x = draft[i];
        outside = outside || static_cast<uint32_t>(x) >= static_cast<uint32_t>(V);
        mark(x);
    }
    for (int32_t i = ru.b0 + tid; i < ru.b1; i += kFewThreads) {
        const int32_t x = u.bias_id[i];
        outside = outside || static_cast<uint32_t>(x) >= static_cast<uint32_t>(V);
        mark(x);
    }
    if (tells) {
        if (__syncthreads_or(outside)) st |= SV_ST_TOKEN_RANGE;
        if (__syncthreads_or(over)) st |= SV_ST_BAD_MASK;
        if (tid == 0) a.status[r] = static_cast<int32_t>(st);
    }
    __syncthreads();

    // how many ids are marked before each word
    const int32_t share = (words + kFewThreads - 1) / kFewThreads, w0 = min(tid * share, words), w1 = min(w0 + share, words);
    int32_t mine = 0;
    for (int32_t w = w0; w < w1; ++w) mine += __popc(s_bits[w]);
    int32_t before = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int32_t o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) s_warp[warp] = before;
    __syncthreads();
    int32_t ids = 0;
    before -= mine;
    for (int w = 0; w < kFewThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        ids += s_warp[w];
    }
    for (int32_t w = w0; w < w1; ++w) {
        s_rank[w] = before;
        before += __popc(s_bits[w]);
    }

    bool streamed = early;
    for (int32_t from = 0; from < ids || !streamed; from += g.table) {
        const int32_t n = max(min(ids - from, g.table), 0);
        for (int32_t i = tid; i < n; i += kFewThreads) {
            s_tab[i] = 0;
            if (biased) s_bias[i] = 0;
        }
        __syncthreads();
        // an id's place in the window, at least n for none
        auto place = [&](int32_t x) -> uint32_t {
            if (static_cast<uint32_t>(x - low) >= span) return 0xFFFFFFFFu;
            const int32_t w = (x - base) >> 5;
            return static_cast<uint32_t>(s_rank[w] + __popc(s_bits[w] & ((1u << (x & 31)) - 1)) - from);
        };
        const uint32_t limit = static_cast<uint32_t>(n);
        for (int32_t w = tid; w < words; w += kFewThreads) {
            uint32_t p = static_cast<uint32_t>(s_rank[w] - from);
            for (uint32_t b = s_bits[w]; b != 0; b &= b - 1, ++p)
                if (p < limit) s_list[p] = 32 * w + __ffs(b) - 1;
        }
        each_token([&](int32_t i, int32_t x) {
            const uint32_t p = place(x);
            if (p >= limit) return;
            if (i >= ru.prompt)
                atomicAdd(&s_tab[p], 1u);
            else
                atomicOr(&s_tab[p], kAdjSeen);
        });
        for (int32_t i = tid; i < g.drafts; i += kFewThreads) {
            const uint32_t p = place(draft[i]);
            if (p >= limit) continue;
            uint32_t old = s_tab[p], was;
            do {
                was = old;
                s_next[i] = static_cast<uint16_t>((was & kAdjHead) >> kAdjHeadShift);
                old = atomicCAS(&s_tab[p], was, (was & ~kAdjHead) | (static_cast<uint32_t>(i + 1) << kAdjHeadShift));
            } while (old != was);
        }
        for (int32_t i = ru.b0 + tid; i < ru.b1; i += kFewThreads) {
            const uint32_t p = place(u.bias_id[i]);
            if (p < limit) atomicMax(&s_bias[p], static_cast<uint32_t>(i) + 1);
        }
        if (!streamed) stream();
        streamed = true;
        __syncthreads();
        for (int32_t j = 0; j < g.rows; ++j) {
            const T* src = in + j * a.in.stride;
            T* dst = out + j * a.out.stride;
            const uint32_t* mask = mask_at(s_row[j]);
            const int32_t start = start_of(dst), end = min(start + g.slice, V);
            const int32_t before_branch = j > 0 ? (j - 1) / a.k * a.k : 0;
            for (int32_t i = tid; i < n; i += kFewThreads) {
                const int32_t x = base + s_list[i];
                if (x < start || x >= end) continue;
                const T raw = src[x];  // on its way while the mask's word is
                if (!allowed(mask, x)) continue;
                const uint32_t word = s_tab[i], entry = biased ? s_bias[i] : 0u;
                uint32_t count = word & kAdjCount;
                for (uint32_t e = (word & kAdjHead) >> kAdjHeadShift; e != 0; e = s_next[e - 1])
                    count += static_cast<int32_t>(e) > before_branch && static_cast<int32_t>(e) <= j;
                dst[x] = adjust<T>(raw, (word & kAdjSeen) != 0, count, entry != 0 ? &u.bias_value[entry - 1] : nullptr, ru);
            }
        }
        __syncthreads();
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

// Whether a call's requests have few rows, and are so many that the other kernel's blocks would not all be resident at
// once: 16 requests of one row take 9.0 us with that one and 9.6 with this (in place 7.2 and 8.7), 24 take 10.1 and 10.2 (10.7
// and 8.7), 64 30 and 20 (25 and 15).
bool few_rows(const AdjustArgs& a, const AdjustGeom& g)
{
    return g.rows <= (a.in.data == a.out.data ? kFewRowsInPlace : kFewRows) &&
           static_cast<int64_t>(a.R) * g.slices > 4 * std::max(1, device_sm_count());
}

FewGeom few_geom_of(const AdjustArgs& a)
{
    const int sms = std::max(1, device_sm_count());
    FewGeom g{};
    g.drafts = a.branches * a.k;
    g.rows = 1 + g.drafts;
    const int64_t ids = static_cast<int64_t>(a.in.width) + kAdjEdge - 1, span = kFewVecs * 32 * 8;  // a warp's vectors of bf16
    const int64_t resident = std::max<int64_t>(1, kFewBlocks * sms / a.R);  // slices of a row
    const int64_t slices = std::max((ids + kFewSlice - 1) / kFewSlice, std::min(resident, (ids + kFewLeast - 1) / kFewLeast));
    g.slice = static_cast<int32_t>(((ids + slices - 1) / slices + span - 1) / span * span);
    g.slices = static_cast<int32_t>((ids + g.slice - 1) / g.slice);
    const int64_t met = static_cast<int64_t>(a.rules.history != nullptr ? a.rules.history_width : 0) + g.drafts + a.rules.bias_entries;
    g.table = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({met, g.slice + kAdjEdge, kFewTable})));
    return g;
}

}  // namespace

bool adjust_fits(const AdjustArgs& a)
{
    const AdjustGeom g = geom_of(a);
    if (few_rows(a, g)) return static_cast<int64_t>(a.R) * few_geom_of(a).slices <= INT32_MAX;
    return static_cast<int64_t>(a.R) * g.slices * g.groups <= INT32_MAX;
}

cudaError_t launch_adjust_logits(const AdjustArgs& a, cudaStream_t stream)
{
    const bool tiles = by_tiles(a), bf16 = a.in.dtype == SV_BF16;
    const AdjustGeom g = geom_of(a);
    if (few_rows(a, g)) {
        const FewGeom f = few_geom_of(a);
        const int bytes = few_layout(f, a.rules.bias_entries != 0).bytes;
        const bool in_place = a.in.data == a.out.data;
        auto* kernel = in_place ? bf16 ? adjust_few_kernel<uint16_t, Lie::InPlace> : adjust_few_kernel<uint32_t, Lie::InPlace>
                       : tiles  ? bf16 ? adjust_few_kernel<uint16_t, Lie::Alike> : adjust_few_kernel<uint32_t, Lie::Alike>
                                : bf16 ? adjust_few_kernel<uint16_t, Lie::Apart> : adjust_few_kernel<uint32_t, Lie::Apart>;
        if (cudaError_t e = allow_shared(kernel, bytes)) return e;
        kernel<<<static_cast<unsigned>(static_cast<int64_t>(a.R) * f.slices), kFewThreads, bytes, stream>>>(a, f);
        return cudaGetLastError();
    }
    const int bytes = layout_of(g, tiles).bytes;
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.R) * g.slices * g.groups);
    auto* kernel = tiles ? bf16 ? adjust_kernel<uint16_t, true> : adjust_kernel<uint32_t, true>
                         : bf16 ? adjust_kernel<uint16_t, false> : adjust_kernel<uint32_t, false>;
    if (cudaError_t e = allow_shared(kernel, bytes)) return e;
    kernel<<<blocks, kAdjThreads, bytes, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
