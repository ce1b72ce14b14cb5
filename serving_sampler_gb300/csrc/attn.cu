// sv_tree_attention: out = softmax(scale q k^T) v of a step's tokens over the paged
// cache, on the tensor cores.
//
// Rows.  The query heads that share a key head see the same keys, so a tile of 128
// rows holds 128 / G tokens with their G heads each (row = token * G + head).  Keys
// come in tiles of 128: S = Q K^T, P = 2^(c S - m), O += P V, c = |scale| log2 e
// (a negative scale turns the sign of Q inside the product).
//
// One persistent CTA per SM, warp roles:
//   warps 0, 2  copy K and V tiles, block by block, with tensor maps into a ring of
//               stages (the block ids of the next tile are fetched before the wait for
//               a stage);
//   warp 1      issues the products; S in tensor memory, P over S in tensor memory as
//               the left operand of P V, O in tensor memory;
//   warp 3      lists the CTA's runs of work for the others, copies Q, and cleans V where a
//               tile holds positions that not every row sees: rows behind the last key
//               become 0 (P is 0 there, but 0 * NaN is not), and so do NaN and infinite
//               entries, which are noted and added in 32 bits at the end of the group to
//               the rows that do see them;
//   warps 4-7, 8-11   two streams of softmax, one row per thread; each stream has an S and
//               an O of its own, so that while one's softmax runs the other's products do.
//
// Streams.  Where a request's rows fit one tile the streams split its keys: of a group's
// tiles the even ones go to stream 0 and the odd ones to stream 1, and at the group's end
// each warpgroup joins half of the columns of both.  Where a request has more rows the
// streams are two row tiles that use the same K and V from shared memory.
//
// Order of sums.  A request's keys are cut into groups of whole tiles by a rule on
// its own lengths (request_of).  Within a group a stream's O and sum l belong to a
// reference m, the row maximum of its first tile; a later tile's maximum replaces it
// only when it is more than 2^8 above (O is then rescaled), which no 32-bit sum
// notices.  (O, l, m) and (O', l', m') are joined at max(m, m'): the streams of a
// group, then the groups from the first to the last.  A CTA that has an item from its
// first group on joins as it goes; other groups go to the workspace and
// attn_join_kernel joins them in the same order with the same instructions, so the bits
// do not depend on where the work was cut.  The sums so far stand in registers, half a
// row in a thread; with several row tiles a thread has a whole row, whose 128 registers
// left the softmax too few (292 us for 64 x 65 tokens, with spills), so they stand in
// the workspace, which L2 holds, where the thread alone reads and writes them (221 us).
//
// Work.  An item is (request, key head, row tile or pair of them), a unit one group of
// an item.  All units lie on one line, in cost of two per tile, two per group and eight
// per item, cut evenly over the CTAs; every CTA finds its share itself from the lengths
// on the device.
//
// What bounds it (heads of 128 in bf16 unless said otherwise, time of the kernel, GB300):
//   64 x 9 tokens, 4 heads to a key head, 4,250 keys on average: bytes.  200 us for the
//   1.2 GB of K and V, 6.0 TB/s, 0.88 of a copy's rate.
//   64 x 65 tokens, 7 heads to a key head, 2,500 keys: the waits in the chain of a row tile,
//   product, softmax, product, of which two alternate, and the joining of groups (a fifth of
//   the time).  191 us, 0.40 of the rate of a plain matrix product, with the tensor pipe active
//   42 % of it, exponentials 18 % and memory at 55 %.
//   17 x 33 tokens, one head to a key head, 64 entries in fp16, 1,700 keys: the same chain,
//   as a tile's rows are 33; and 5 us before the first product.  41 us.
//   9 tokens over 131,071 keys: bytes, 86 us, 6.2 TB/s, and 12 us for the join.
//   One token, 777 keys: latency, two launches and a chain of loads, 10 us and 5.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_internal.h"
#include "sv_tensor.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;       // rows of a row tile, keys of a key tile
constexpr int kMaxStages = 12;
// Tensor memory: S of the two streams, then O.  Heads of 64 leave room for a second O of each
// stream, so that a group's products need not wait until the group before has been read.
template <int DP>
constexpr int kSums = DP == 64 ? 2 : 1;
template <int DP>
__device__ __forceinline__ uint32_t o_column(uint32_t group, int s)
{
    return 2 * kTile + (kSums<DP> == 2 ? (group & 1u) * 2 * DP : 0u) + s * DP;
}
constexpr int kAttnThreads = 384;
constexpr size_t kMaxShared = 232448;  // bytes of shared memory a CTA can have
constexpr int kRunRing = 4;       // runs that are listed at a time
constexpr int kRunReaders = 11;   // warps that read them: two that copy, the products, eight of softmax
constexpr int kGroupRing = 16;   // groups whose notes of non-finite values are kept
constexpr float kGrow = 8.0f;    // log2 by which a tile's maximum may pass the reference

// Where a CTA's share begins: a group of an item of a request.
struct Start {
    int32_t r, item, g, pad;
};
__device__ __forceinline__ bool before(const Start& a, const Start& b)
{
    return a.r != b.r ? a.r < b.r : a.item != b.item ? a.item < b.item : a.g < b.g;
}

struct alignas(16) Request {
    int32_t tok0, na, kv, ctx;  // first token, tokens that attend, keys, keys before the tokens
    int32_t tiles, per_head;    // row tiles, items of a key head
    int32_t gt, ng, cost;       // key tiles of a group, groups and cost of an item over all keys
};

struct AttnParams {
    const int32_t *block_table, *kv_len, *cu_tokens;
    const uint32_t* mask;
    int32_t R, T, max_blocks, max_kv, max_tokens, mask_words;
    Divisor by_block, by_tile, by_sms;  // block_size, tile_tokens, sms
    int32_t wave;                       // items of a key head for every SM to have one, of one row tile or two
    int32_t block_size, num_blocks, kv_heads, group, tile_tokens, head_dim;
    int32_t box_tokens;  // tokens a copy of Q brings
    int32_t q_chunk;     // bytes of 64 columns of Q
    int32_t box_rows;  // rows one copy brings: they divide a block and a tile
    int32_t stages, sms;
    float c;
    uint32_t word_qk, word_pv;
    const uint16_t* v;
    int64_t block_stride, token_stride, head_stride;
    uint16_t* out;
    int64_t out_token_stride, out_head_stride;
    float* lse;
    int32_t* status;
    Start* starts;    // [CTAs + 1]
    Request* firsts;  // [CTAs]: the request that a share begins in (looked at where it begins inside an item)
    uint32_t* flags;  // [CTAs]
    // [CTAs][slots_per_cta]: O as [DP / 4][rows][4], then m [rows], l [rows].  Slot 0: what the CTA's
    // last item has, and, with several row tiles, the sums of the run at hand
    float* slots;
    int64_t slot_floats;
    int32_t slots_per_cta, slot_rows;
    int32_t stop_cta;  // a CTA that gives up at its first wait (self-test; -1: none)
};

// A request's lengths as they come, loaded before they are looked at.
struct Lengths {
    int32_t t0, t1, kv;
};
__device__ __forceinline__ Lengths lengths_of(const AttnParams& p, int32_t r)
{
    return Lengths{p.cu_tokens[r], p.cu_tokens[r + 1], p.kv_len[r]};
}

// Groups.  Few and long ones cost least (a group's end is a pass over O and leaves the
// products idle); many and short ones let a request alone fill the machine.  A group has
// about one and a half times the square root of the item's tiles, at least 2 (8 where two
// row tiles share them: with 16, 64 x 65 tokens over 2,500 keys take 201 us instead of 218,
// but 4 x 65 take 49 instead of 37 and a request alone 46 instead of 33); where
// that is near, the number that gives a request alone one or two units for every SM; and
// an even number, so that a tile's stream is its parity.
__device__ __forceinline__ Request request_from(const AttnParams& p, const Lengths& x)
{
    Request q;
    const int32_t t0 = min(max(x.t0, 0), p.T), t1 = min(max(x.t1, t0), p.T);
    q.tok0 = t0;
    q.na = min(t1 - t0, p.max_tokens);
    q.kv = min(max(x.kv, 0), p.max_kv);
    q.ctx = q.kv - (t1 - t0);
    q.tiles = p.by_tile.quotient(q.na + p.tile_tokens - 1);
    q.per_head = (q.tiles + 1) / 2;
    const int32_t nt = (q.kv + kTile - 1) / kTile;
    const int32_t wave = q.per_head <= 1 ? p.wave : max(1, p.sms / (p.kv_heads * q.per_head));
    const int32_t root = 2 * static_cast<int32_t>(0.75f * sqrtf(static_cast<float>(nt)));
    const int32_t one = (nt + wave - 1) / wave, two = (nt + 2 * wave - 1) / (2 * wave);
    const int32_t even = 5 * two >= 4 * root ? two : 5 * one >= 4 * root ? one : root;
    q.gt = (max(q.tiles > 1 ? 8 : 2, even) + 1) & ~1;
    q.ng = max(1, (nt + q.gt - 1) / q.gt);
    q.cost = 2 * nt + 2 * q.ng + 8;
    return q;
}
__device__ __forceinline__ Request request_of(const AttnParams& p, int32_t r)
{
    return request_from(p, lengths_of(p, r));
}

// An item's groups that lie in a CTA's share.
struct Run {
    int32_t r;                      // request, -1 behind the last run
    int32_t tok0, na, ctx, kv_end;  // keys [0, kv_end) are looked at
    int32_t head, tile;             // key head, (first) row tile
    bool split, second;             // the streams split the keys; a second row tile
    int32_t gt, ga, gb, ng;         // tiles of a group, groups [ga, gb) of ng
    int32_t nt;                     // key tiles of the item
};

struct Walk {
    Start at, end;
    int32_t known;
    Request q;
};

__device__ __forceinline__ int32_t item_tiles(const AttnParams& p, const Request& q, int32_t tile, int32_t* kv_end)
{
    int32_t e = q.kv;
    if (p.mask == nullptr) e = min(e, q.ctx + min(q.na, (tile + 2) * p.tile_tokens));
    *kv_end = max(e, 0);
    return (*kv_end + kTile - 1) / kTile;
}

__device__ __forceinline__ bool next_run(const AttnParams& p, Walk& w, Run& out)
{
    while (before(w.at, w.end)) {
        if (w.known != w.at.r) {
            w.q = request_of(p, w.at.r);
            w.known = w.at.r;
        }
        const Request& q = w.q;
        if (w.at.item >= q.per_head * p.kv_heads) {
            w.at = Start{w.at.r + 1, 0, 0, 0};
            continue;
        }
        out.head = w.at.item / q.per_head;
        out.tile = 2 * (w.at.item - out.head * q.per_head);
        out.nt = item_tiles(p, q, out.tile, &out.kv_end);
        out.ng = max(1, (out.nt + q.gt - 1) / q.gt);
        out.ga = w.at.g;
        out.gb = w.end.r == w.at.r && w.end.item == w.at.item ? min(out.ng, w.end.g) : out.ng;
        w.at.item += 1;
        w.at.g = 0;
        if (out.ga >= out.gb) continue;
        out.r = w.at.r;
        out.tok0 = q.tok0;
        out.na = q.na;
        out.ctx = q.ctx;
        out.gt = q.gt;
        out.split = q.tiles == 1;
        out.second = out.tile + 1 < q.tiles;
        return true;
    }
    return false;
}

// Positions below this are seen by every row from row tile `tile` on.
__device__ __forceinline__ int32_t seen_by_all(const AttnParams& p, const Run& u, int32_t tile)
{
    return min(p.mask != nullptr ? u.ctx : u.ctx + tile * p.tile_tokens + 1, u.kv_end);
}

// A position of the ring of stages.
struct Ring {
    int32_t stage;
    uint32_t phase;
    __device__ __forceinline__ void next2(int32_t n)
    {
        stage += 2;
        if (stage >= n) {
            stage -= n;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void prev2(int32_t n)
    {
        stage -= 2;
        if (stage < 0) {
            stage += n;
            phase ^= 1u;
        }
    }
};

struct Shared {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t q_full[2], q_empty[2];              // by buffer
    uint64_t s_full[2], p_full[2], pv_done[2];   // by stream, a phase per tile
    uint64_t g_done, o_free[2];                  // a phase per group whose keys are split (o_free: of every other)
    uint64_t run_full[kRunRing], run_empty[kRunRing];
    uint64_t drain;
    Run runs[kRunRing];
    uint64_t v_ok[kMaxStages];  // the stage's V has been cleaned
    int64_t scan[16];
    Start start, end;
    Request first;  // request first_r, which the share begins in or behind
    int32_t first_r;
    float ref[2][kTile], sum[2][kTile];  // of a stream's group, by row
    uint32_t tmem;
    uint32_t odd[kGroupRing];  // 1 + number of the group whose V had non-finite entries
    int stop;
};

// Bounded wait; gives up as well when another role of the CTA has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Shared& sh)
{
    if (mbar_poll(bar, parity)) return true;
    const long long t0 = clock64();
    volatile int* stop = &sh.stop;
    while (!mbar_poll(bar, parity)) {
        if (*stop != 0) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            *stop = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Shared& sh)
{
    return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, sh)) != 0;
}

// The list of runs, for a warp: one after the other, each given back when nothing of it is
// looked at any more.
struct Runs {
    uint32_t k = 0;
    __device__ __forceinline__ const Run* get(Shared& sh) const
    {
        return warp_wait(&sh.run_full[k % kRunRing], (k / kRunRing) & 1u, sh) ? &sh.runs[k % kRunRing] : nullptr;
    }
    __device__ __forceinline__ void give_back(Shared& sh, uint32_t which) const
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.run_empty[which % kRunRing]);
    }
};

template <bool F16>
__device__ __forceinline__ uint32_t pack_pair(float x, float y)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ float widen(uint16_t w)
{
    return F16 ? __half2float(__ushort_as_half(w)) : __uint_as_float(static_cast<uint32_t>(w) << 16);
}

// Factors that bring two groups' sums to the larger of their references.
struct Join {
    float m, a, b;
};
__device__ __forceinline__ Join join_at(float m, float mg)
{
    Join j;
    j.m = fmaxf(m, mg);
    j.a = m == j.m ? 1.0f : exp2_fast(m - j.m);
    j.b = mg == j.m ? 1.0f : exp2_fast(mg - j.m);
    return j;
}
__device__ __forceinline__ float join_sum(float x, float y, const Join& j)
{
    return __fmaf_rn(y, j.b, __fmul_rn(x, j.a));
}
// the same on two entries at once: the two roundings are those of join_sum
__device__ __forceinline__ float2 join_sum2(float2 x, float2 y, const Join& j)
{
    return fma2(y, make_float2(j.b, j.b), mul2(x, make_float2(j.a, j.a)));
}
__device__ __forceinline__ float final_lse(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// ---- shares -------------------------------------------------------------------
// Locate the unit whose start is nearest to `at` on the line, inside request r whose
// costs begin at `first`.  (The next one behind would give two groups to CTAs whose shares
// are a little more than one: 138 us for 9 tokens over 131,071 keys.)
__device__ __forceinline__ Start locate(const AttnParams& p, const Request& q, int32_t r, int64_t first, int64_t at)
{
    const int64_t off = at - first;
    int32_t item = off <= 0x7FFFFFFF ? static_cast<int32_t>(static_cast<uint32_t>(off) / static_cast<uint32_t>(q.cost))
                                     : static_cast<int32_t>(off / q.cost);
    const int32_t in = static_cast<int32_t>(off - static_cast<int64_t>(item) * q.cost);
    int32_t g = static_cast<int32_t>(static_cast<uint32_t>(in + q.gt + 1) / static_cast<uint32_t>(2 * q.gt + 2));
    if (g >= q.ng) {
        g = 0;
        ++item;
    }
    if (item >= q.per_head * p.kv_heads) return Start{r + 1, 0, 0, 0};
    return Start{r, item, g, 0};
}

__device__ __forceinline__ int64_t request_cost(const AttnParams& p, const Request& q)
{
    return static_cast<int64_t>(q.per_head) * p.kv_heads * q.cost;
}

// Every thread of the CTA; sets sh.start, sh.first and sh.end.  `x`: the lengths of request
// threadIdx.x.  On the way of every call, so kept short: one pass where there is a thread for every
// request, and no 64-bit division (1.7 us less for every call).
__device__ void find_share(const AttnParams& p, Shared& sh, const Lengths& x)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    // Request r0 + tid and where its costs begin; `base` becomes where the next requests' do.
    Request q{};
    int64_t cost = 0, first = 0, base = 0, total = 0;
    auto take = [&](int32_t r0) {
        const int32_t r = r0 + tid;
        cost = 0;
        if (r < p.R) {
            q = request_from(p, r0 == 0 ? x : lengths_of(p, r));
            cost = request_cost(p, q);
        }
        int64_t sum = cost;
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += u;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = sum;
        __syncthreads();
        first = base + sum - cost;
#pragma unroll 1
        for (int w = 0; w < warps; ++w) {
            if (w < warp) first += sh.scan[w];
            base += sh.scan[w];
        }
    };
    if (tid == 0) {
        sh.start = sh.end = Start{p.R, 0, 0, 0};
        sh.first_r = -1;
    }
    // Twice over the requests, of which the first time is for the total; where there is a thread for each
    // of them, once.
    const int32_t rounds = (p.R + nt - 1) / nt;
    int64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int32_t k = rounds > 1 ? 0 : 1; k < 2 * rounds; ++k) {
        if (k == rounds) base = 0;
        take((k < rounds ? k : k - rounds) * nt);
        if (k == (rounds > 1 ? rounds - 1 : 1)) {
            total = base;
            // total * c / grid
            const int32_t c = static_cast<int32_t>(blockIdx.x), grid = static_cast<int32_t>(gridDim.x);
            const int64_t each = total <= 0x7FFFFFFF ? p.by_sms.quotient(static_cast<int32_t>(total)) : total / grid;
            const int32_t rest = static_cast<int32_t>(total - each * grid);
            lo = each * c + p.by_sms.quotient(rest * c);
            hi = each * (c + 1) + p.by_sms.quotient(rest * (c + 1));
        }
        if (k < rounds) continue;
        const int32_t r = (k - rounds) * nt + tid;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const int64_t at = side == 0 ? lo : hi;
            if (at < first || at >= first + cost) continue;
            const Start found = locate(p, q, r, first, at);
            if (side == 0) {
                sh.start = found;
                sh.first = q;
                sh.first_r = r;
            } else {
                sh.end = found;
            }
        }
    }
    __syncthreads();
}

// ---- warps 0 and 2: K and V --------------------------------------------------------
// Tile t of the line fills stages 2 t (K) and 2 t + 1 (V) of the ring, whose number of stages
// is even: K and V have stages of their own.  Warp 0 copies K and warp 2 V (one warp for both
// could not issue the copies of 16-token blocks fast enough).  Lane i copies box i.
template <int DP>
__device__ void copy_tiles(const AttnParams& p, Shared& sh, unsigned char* ring, const CUtensorMap* map, int first)
{
    constexpr int kChunks = DP / 64;
    constexpr uint32_t kStage = kTile * DP * 2;
    const int lane = threadIdx.x & 31;
    Runs runs;
    Ring rt{first, 0};
    int32_t fills = 0;  // of this warp; from the ring's second turn on a stage is waited for
    bool ok = true;
    const int32_t subs = kTile / p.box_rows;
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * 128u;
    for (; ok; ++runs.k) {
        const Run* const next = runs.get(sh);
        ok = next != nullptr;
        if (!ok || next->r < 0) break;
        const Run u = *next;
        runs.give_back(sh, runs.k);
        const int32_t* table = p.block_table + static_cast<int64_t>(u.r) * p.max_blocks;
        const int32_t t1 = min(u.gb * u.gt, u.nt);
        int32_t t = u.ga * u.gt;
        if (t >= t1) continue;
        auto block_of = [&](int32_t tile) -> int32_t {
            const int32_t x = tile * kTile + lane * p.box_rows;
            return lane < subs && x < u.kv_end ? table[p.by_block.quotient(x)] : 0;
        };
        int32_t id = block_of(t);
        for (; t < t1; ++t) {
            const int32_t block = id, x0 = t * kTile;
            if (t + 1 < t1) id = block_of(t + 1);  // in flight while this tile is issued
            const int32_t at = x0 + lane * p.box_rows, place = at - p.by_block.quotient(at) * p.block_size;
            const int32_t live = min(subs, (u.kv_end - x0 + p.box_rows - 1) / p.box_rows);
            uint64_t* full = &sh.kv_full[rt.stage];
            // the stage's fill before this one is the ring's last turn: `first + 2 * fills` stages in
            if (first + 2 * fills >= p.stages && !warp_wait(&sh.kv_empty[rt.stage], rt.phase ^ 1u, sh)) {
                ok = false;
                break;
            }
            unsigned char* dst = ring + static_cast<size_t>(rt.stage) * kStage;
            if (elect_one()) mbar_arrive_expect_tx(full, static_cast<uint32_t>(live) * box_bytes * kChunks);
            __syncwarp();
            if (lane < live) {
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch)
                    tma_load_4d(dst + lane * box_bytes + ch * kTile * 128, map, full, ch * 64, place, u.head, block);
            }
            __syncwarp();
            fills = min(fills + 1, 1 << 20);
            rt.next2(p.stages);
        }
    }
    // a CTA that gave up does not leave before its copies have landed: the last fill of each of the copier's stages
    if (!ok || sh.stop != 0) {
        for (int32_t i = min(fills, p.stages / 2); i > 0; --i) {
            rt.prev2(p.stages);
            mbar_wait_bounded(&sh.kv_full[rt.stage], rt.phase);
        }
    }
}

// ---- warp 3: Q, and V that not every row sees ---------------------------------------
// The warp follows every stage, also those it has nothing to do with, and each stage
// waits for its arrival before it is filled again: the parity of a barrier tells two
// fills of a stage apart only for a warp that is never a whole turn of the ring ahead
// or behind.
template <int DP, bool F16, bool MULTI>
__device__ void copy_q_clean_v(const AttnParams& p, Shared& sh, unsigned char* q_smem, unsigned char* ring,
                               const CUtensorMap* mq)
{
    constexpr int kChunks = DP / 64;
    constexpr uint32_t kStage = kTile * DP * 2;
    constexpr uint32_t kExp = F16 ? 0x7C007C00u : 0x7F807F80u;
    const int lane = threadIdx.x & 31;
    Walk w{sh.start, sh.end, sh.first_r, sh.first};
    Ring rk{0, 0}, rv{1, 0};
    uint32_t groups = 0, listed = 0, q_runs = 0, used[2] = {0, 0};
    bool more = true;  // runs to list
    const uint32_t q_bytes = static_cast<uint32_t>(p.group * p.box_tokens * 128 * kChunks);
    // Lists the next run, or the list's end.
    auto list = [&]() {
        if (listed >= kRunRing && !warp_wait(&sh.run_empty[listed % kRunRing], (listed / kRunRing - 1) & 1u, sh)) return false;
        Run u;
        more = next_run(p, w, u);
        if (!more) u = Run{-1};  // the softmax reads the rest of it too: one turn, no tile
        if (lane == 0) {
            sh.runs[listed % kRunRing] = u;
            mbar_arrive(&sh.run_full[listed % kRunRing]);
        }
        __syncwarp();
        ++listed;
        return true;
    };
    // Q of a run
    auto copy_q = [&](const Run& u) {
        for (int i = 0; i < (u.second ? 2 : 1); ++i) {
            const int b = MULTI ? i : q_runs & 1;
            if (used[b] > 0 && !warp_wait(&sh.q_empty[b], (used[b] - 1) & 1u, sh)) return false;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sh.q_full[b], q_bytes);
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch)
                    tma_load_3d(q_smem + (b * kChunks + ch) * p.q_chunk, mq, &sh.q_full[b], ch * 64, u.head * p.group,
                                u.tok0 + (u.tile + i) * p.tile_tokens);
            }
            __syncwarp();
            ++used[b];
        }
        ++q_runs;
        return true;
    };
    // Two runs are listed ahead of the one that is followed: a slot of the list is free again when the
    // softmax of the run after it has begun, which needs no more than the runs followed so far.  With two
    // buffers Q is a run ahead too.  (Two row tiles take both; their Q is waited for by products that
    // this warp's work on the run comes before, so it cannot be ahead.)
    bool ok = true;
    uint32_t copied = 0;  // runs whose Q is (not MULTI)
    for (uint32_t k = 0; ok; ++k) {
#pragma unroll 1
        while (ok && more && listed < k + 3) {
            ok = list();
            const Run& v = sh.runs[copied % kRunRing];
            if (ok && !MULTI && copied < k + 2 && copied < listed && v.r >= 0) {
                if (v.nt > 0) ok = copy_q(v);
                ++copied;
            }
        }
        const Run u = sh.runs[k % kRunRing];
        if (!ok || u.r < 0) break;
        if (MULTI && u.nt > 0) ok = copy_q(u);
        if (!ok) break;
        const int32_t t1 = min(u.gb * u.gt, u.nt);
        if (u.ga * u.gt >= t1) continue;
        const int32_t all = seen_by_all(p, u, u.tile);
        for (int32_t t = u.ga * u.gt; ok && t < t1; ++t) {
            const int32_t x0 = t * kTile;
            ok = warp_wait(&sh.kv_full[rk.stage], rk.phase, sh);
            if (!ok) break;
            if (lane == 0) mbar_arrive(&sh.kv_empty[rk.stage]);
            ok = warp_wait(&sh.kv_full[rv.stage], rv.phase, sh);
            if (!ok) break;
            if (x0 + kTile > all) {
                unsigned char* base = ring + static_cast<size_t>(rv.stage) * kStage;
                const int32_t first = max(0, all - x0), end = min(kTile, u.kv_end - x0);
                bool odd = false;
                for (int32_t v = first * 8 + lane; v < kTile * 8; v += 32) {
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch) {
                        uint4* at = reinterpret_cast<uint4*>(base + ch * kTile * 128) + v;
                        if ((v >> 3) >= end) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            const uint4 x = *at;
                            const uint32_t bx = __vcmpeq2(x.x & kExp, kExp), by = __vcmpeq2(x.y & kExp, kExp),
                                           bz = __vcmpeq2(x.z & kExp, kExp), bw = __vcmpeq2(x.w & kExp, kExp);
                            if ((bx | by | bz | bw) != 0) {
                                odd = true;
                                *at = make_uint4(x.x & ~bx, x.y & ~by, x.z & ~bz, x.w & ~bw);
                            }
                        }
                    }
                }
                const uint32_t group = groups + (t / u.gt - u.ga);
                if (__any_sync(0xFFFFFFFFu, odd) && lane == 0) sh.odd[group % kGroupRing] = group + 1;
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.v_ok[rv.stage]);
            }
            if (lane == 0) mbar_arrive(&sh.kv_empty[rv.stage]);
            rk.next2(p.stages);
            rv.next2(p.stages);
        }
        groups += u.gb - u.ga;
    }
    if (!ok || sh.stop != 0)  // the copies of Q that were issued
        for (int b = 0; b < 2; ++b)
            if (used[b] > 0) mbar_wait_bounded(&sh.q_full[b], (used[b] - 1) & 1u);
}

// ---- warp 1: products -------------------------------------------------------------------
template <int DP, bool MULTI>
__device__ void issue_products(const AttnParams& p, Shared& sh, uint32_t q_addr, uint32_t ring_addr, uint32_t tmem)
{
    constexpr uint32_t kStage = kTile * DP * 2, kChunk = kTile * 128;
    Runs list;
    Ring rk{0, 0}, rv{1, 0};     // next key tile to multiply with Q, next value tile
    uint32_t tiles[2] = {0, 0};  // by stream
    uint32_t used[2] = {0, 0};   // runs by buffer of Q
    uint32_t groups = 0;         // groups so far,
    uint32_t splits = 0, freed = 0;  // those whose keys are split, and of them the ones seen to be read
    bool after_split = false;    // the group before was one
    uint32_t cleaned = 0;        // a bit per stage: parity of its cleanings
    uint32_t runs = 0;

    auto wait_k = [&]() {
        if (!warp_wait(&sh.kv_full[rk.stage], rk.phase, sh)) return false;
        tmem_fence_after();
        return true;
    };
    auto wait_v = [&](bool clean) {
        if (!clean) return warp_wait(&sh.kv_full[rv.stage], rv.phase, sh);
        if (!warp_wait(&sh.v_ok[rv.stage], (cleaned >> rv.stage) & 1u, sh)) return false;
        cleaned ^= 1u << rv.stage;
        return true;
    };
    // S of stream s = Q[b] K; `free_k`: the tile's last use, `free_q`: the run's
    auto qk = [&](int s, int b, bool free_k, bool free_q) {
        if (elect_one()) {
            const uint64_t qa = smem_operand(q_addr + b * (DP / 64) * p.q_chunk, 16, 1024);
            const uint64_t kb = smem_operand(ring_addr + rk.stage * kStage, 16, 1024);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                product_ss(tmem + s * kTile, qa + (((k / 4) * p.q_chunk + (k % 4) * 32) >> 4),
                           kb + (((k / 4) * kChunk + (k % 4) * 32) >> 4), p.word_qk, k > 0);
            product_commit(&sh.s_full[s]);
            if (free_k) product_commit(&sh.kv_empty[rk.stage]);
            if (free_q) product_commit(&sh.q_empty[b]);
        }
        if (free_k) rk.next2(p.stages);
    };
    // A group's first products write O.  What lay there, of the group before (of the one before that
    // where there are two O), has been read: a warpgroup reads its own stream before it lets the next
    // products begin, and says so where it reads the other's.
    auto begin_group = [&]() {
        const uint32_t need = splits - (kSums<DP> == 2 && after_split ? 1u : 0u);
        for (; freed < need; ++freed)
            if (!warp_wait(&sh.o_free[freed & 1u], (freed >> 1) & 1u, sh)) return false;
        return true;
    };
    auto end_group = [&](bool split) {
        ++groups;
        splits += split;
        after_split = split;
    };
    // O of stream s (+)= P V
    auto pv = [&](int s, bool first, bool free_v) {
        if (!warp_wait(&sh.p_full[s], tiles[s] & 1u, sh)) return false;
        tmem_fence_after();
        if (elect_one()) {
            const uint64_t vb = smem_operand(ring_addr + rv.stage * kStage, kChunk, 1024);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                product_ts(tmem + o_column<DP>(groups, s), tmem + s * kTile + k * 8, vb + ((k * 2048) >> 4), p.word_pv,
                           !first || k > 0);
            product_commit(&sh.pv_done[s]);
            if (free_v) product_commit(&sh.kv_empty[rv.stage]);
        }
        ++tiles[s];
        if (free_v) rv.next2(p.stages);
        return true;
    };

    bool ok = true;
    for (; ok; ++list.k) {
        const Run* const next = list.get(sh);
        ok = next != nullptr;
        if (!ok || next->r < 0) break;
        const Run u = *next;
        list.give_back(sh, list.k);
        const int32_t ta = u.ga * u.gt, tb = min(u.gb * u.gt, u.nt);
        if (ta >= tb) continue;
        const int32_t all = seen_by_all(p, u, u.tile);
        if (!MULTI || u.split) {
            const int b = MULTI ? 0 : runs & 1;
            ok = warp_wait(&sh.q_full[b], used[b] & 1u, sh);
            ++used[b];
            ok = ok && wait_k();
            if (!ok) break;
            qk(0, b, true, ta + 1 == tb);
            if (ta + 1 < tb) {
                ok = wait_k();
                if (!ok) break;
                qk(1, b, true, ta + 2 == tb);
            }
            int32_t in_group = 0;
            for (int32_t t = ta; ok && t < tb; ++t) {
                const int s = t & 1;
                if (in_group == 0) ok = begin_group();
                ok = ok && wait_v((t + 1) * kTile > all) && pv(s, in_group < 2, true);
                if (ok && t + 2 < tb) {
                    ok = wait_k();
                    if (ok) qk(s, b, true, t + 3 == tb);
                }
                if (++in_group == u.gt || t + 1 == tb) {
                    in_group = 0;
                    end_group(true);
                }
            }
        } else {
            const int rows = u.second ? 2 : 1;
            for (int s = 0; s < rows; ++s) {
                ok = ok && warp_wait(&sh.q_full[s], used[s] & 1u, sh);
                ++used[s];
            }
            ok = ok && wait_k();
            if (!ok) break;
            for (int s = 0; s < rows; ++s) qk(s, s, s + 1 == rows, ta + 1 == tb);
            int32_t in_group = 0;
            for (int32_t t = ta; ok && t < tb; ++t) {
                if (in_group == 0) ok = begin_group();
                for (int s = 0; ok && s < rows; ++s) {
                    if (s == 0) ok = wait_v((t + 1) * kTile > all);
                    ok = ok && pv(s, in_group == 0, s + 1 == rows);
                    if (ok && t + 1 < tb) {
                        if (s == 0) ok = wait_k();
                        if (ok) qk(s, s, s + 1 == rows, t + 2 == tb);
                    }
                }
                if (++in_group == u.gt || t + 1 == tb) {
                    in_group = 0;
                    end_group(false);
                }
            }
        }
        ++runs;
    }
    if (!ok || sh.stop != 0) {  // the products that were issued end before tensor memory is given back
        if (elect_one()) product_commit(&sh.drain);
        mbar_wait_bounded(&sh.drain, 0);
    }
}

// ---- warps 4 to 11: softmax, sums, results ---------------------------------------------------
// The 32 positions from x on that token i of the run sees, as bits.
__device__ __forceinline__ uint32_t seen_bits(const AttnParams& p, const Run& u, int32_t i, const uint32_t* words,
                                              int32_t x)
{
    auto below = [](int32_t n) -> uint32_t { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
    if (p.mask == nullptr) return below(min(u.ctx + i + 1, u.kv_end) - x);
    const int32_t j = x - u.ctx;  // the request's token at position x
    auto word = [&](int32_t w) -> uint32_t { return w >= 0 && w < p.mask_words ? words[w] : 0u; };
    uint32_t bits;
    if (j >= 0)
        bits = __funnelshift_r(word(j >> 5), word((j >> 5) + 1), j & 31);
    else if (j <= -32)
        bits = 0xFFFFFFFFu;
    else
        bits = below(-j) | (word(0) << -j);
    return bits & below(u.kv_end - x);
}

// A row's probabilities of a whole tile, P = 2^(c z - m), and their sum, in a loop that is
// not unrolled.  For 64 x 9 tokens over 4,250 keys the loop took 200 us, two steps at a time
// 206, and 222 unrolled with the next scores loaded ahead: the more code, the slower, as the
// warps' roles share one instruction cache.  32 columns a step instead of 16 gave 52 -> 50 us
// for 17 x 33 tokens, loading the next ones ahead in the loop nothing more.  P lies over
// scores that have been read.  It is rounded to the cache's type, as a product takes 16-bit operands,
// and the sum is taken before that: the output's error against 64 bits is 1.05 to 1.4 times that of
// 32-bit probabilities (0.0023 instead of 0.0017 in bf16, 0.00024 instead of 0.00021 in fp16).
template <bool F16>
__device__ __forceinline__ float exp_tile(uint32_t s_addr, float c, float off)
{
    const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
    constexpr int kWide = 32;
    float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
#pragma unroll 1
    for (int step = 0; step < kTile / kWide; ++step) {
        uint32_t z[kWide], pk[kWide / 2];
        tmem_ld(z, s_addr + step * kWide);
        tmem_wait_ld(z);
#pragma unroll
        for (int e = 0; e < kWide / 2; ++e) {
            float2 x = fma2(make_float2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])), c2, off2);
            x.x = exp2_fast(x.x);
            x.y = exp2_fast(x.y);
            if (e & 1)
                s1 = add2(s1, x);
            else
                s0 = add2(s0, x);
            pk[e] = pack_pair<F16>(x.x, x.y);
        }
        tmem_st(s_addr + step * (kWide / 2), pk);
    }
    s0 = add2(s0, s1);
    return s0.x + s0.y;
}

// One stream's state of a row within a group.
struct RowState {
    float ref, off, l;  // reference (as it comes from the product, and scaled) and sum
};

// The softmax of one tile of a stream: scores out, probabilities in their place.
// Returns false when a wait gave up.
template <int DP, bool F16>
__device__ __forceinline__ bool softmax_tile(const AttnParams& p, Shared& sh, const Run& u, int s, uint32_t s_addr,
                                             uint32_t o_addr, int32_t t, bool first, uint32_t n, int32_t all, bool live,
                                             int32_t mine, const uint32_t* words, RowState& st)
{
    const float c = p.c;
    const int32_t x0 = t * kTile;
    const bool masked = x0 + kTile > all;
    float top = -INFINITY;
    if (masked) {  // hidden scores become -inf where they stand
#pragma unroll 1
        for (int ch = 0; ch < 8; ++ch) {
            const uint32_t bits = live ? seen_bits(p, u, mine, words, x0 + (ch & ~1) * 16) >> (16 * (ch & 1)) : 0u;
            uint32_t z[16];
            tmem_ld(z, s_addr + ch * 16);
            tmem_wait_ld(z);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                z[e] = (bits >> e) & 1u ? z[e] : 0xFF800000u;
                top = fmaxf(top, __uint_as_float(z[e]));
            }
            tmem_st(s_addr + ch * 16, z);
        }
        tmem_wait_st();
    } else {
#pragma unroll 1
        for (int col = 0; col < kTile; col += 64) top = fmaxf(top, tmem_max64(s_addr + col));
    }
    if (first) {
        st.ref = top;
    } else {
        const bool grow = live && top > st.ref && (st.ref == -INFINITY || (top - st.ref) * c > kGrow);
        if (__any_sync(0xFFFFFFFFu, grow)) {
            float f = 1.0f;
            if (grow) {
                f = st.ref == -INFINITY ? 0.0f : exp2_fast((st.ref - top) * c);
                st.ref = top;
            }
            st.l *= f;
            // this tile's scores follow the product of the tile before last, so the barrier is not a
            // phase behind the one that is waited for
            if (!warp_wait(&sh.pv_done[s], (n - 1) & 1u, sh)) return false;
            tmem_fence_after();
#pragma unroll 1
            for (int ch = 0; ch < DP / 16; ++ch) {
                uint32_t z[16];
                tmem_ld(z, o_addr + ch * 16);
                tmem_wait_ld(z);
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(__uint_as_float(z[e]) * f);
                tmem_st(o_addr + ch * 16, z);
            }
        }
    }
    st.off = st.ref == -INFINITY ? 0.0f : st.ref * c;
    st.l += exp_tile<F16>(s_addr, c, st.off);
    tmem_wait_st();
    return true;
}

// Non-finite values that were taken out of V join the sums of the rows that see them: those of
// group g, of which the ones whose tile belongs to the stream.
template <int DP, bool F16>
__device__ __noinline__ void add_odd(const AttnParams& p, const Run& u, int32_t g, uint32_t o_addr, int s)
{
    const int row = threadIdx.x & (kTile - 1), token = row / p.group;
    const int32_t i = (u.tile + (u.split ? 0 : s)) * p.tile_tokens + token;
    const int32_t ta = g * u.gt, x0 = max(ta * kTile, seen_by_all(p, u, u.tile));
    const int32_t x1 = min(min(ta + u.gt, u.nt) * kTile, u.kv_end);
    const int32_t* table = p.block_table + static_cast<int64_t>(u.r) * p.max_blocks;
    // a row that is none sees what it may: its sums are not used
    const uint32_t* words =
        p.mask == nullptr ? nullptr : p.mask + static_cast<int64_t>(min(u.tok0 + i, p.T - 1)) * p.mask_words;
#pragma unroll 1
    for (int ch = 0; ch < DP / 16; ++ch) {
        uint32_t z[16];
        tmem_ld(z, o_addr + ch * 16);
        tmem_wait_ld(z);
#pragma unroll 1
        for (int32_t x = x0; x < x1; ++x) {
            if (u.split && ((x / kTile - ta) & 1) != s) continue;
            if (!(seen_bits(p, u, i, words, x) & 1u)) continue;
            const int32_t blk = table[x / p.block_size];
            if (blk < 0 || blk >= p.num_blocks) continue;
            const uint16_t* v = p.v + blk * p.block_stride + (x % p.block_size) * p.token_stride + u.head * p.head_stride +
                                ch * 16;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if (ch * 16 + e < p.head_dim) {
                    const float y = widen<F16>(v[e]);
                    if (!isfinite(y)) z[e] = __float_as_uint(__uint_as_float(z[e]) + y);
                }
            }
        }
        __syncwarp();
        tmem_st(o_addr + ch * 16, z);
    }
    tmem_wait_st();
}

// What is left to do for a stream's last group when its products are complete: it is joined, and
// what the run has is written.  That waits until the first scores of the next group have been
// worked on, so that the products, the other stream and the stores run beside them.
struct Left {
    bool any, split, both, tiles, live, warp_live, whole, last, complete;
    uint32_t run;  // number of its run
    int32_t g;
    int32_t slot;  // of a group that is joined elsewhere
    int32_t t, h;  // the row's token and head
    float mg, lg;
};

template <int DP, bool F16, bool MULTI>
__device__ void softmax_rows(const AttnParams& p, Shared& sh, uint32_t tmem, int s)
{
    constexpr int kHalf = DP / 2;            // columns of O that a warpgroup joins when the keys are split
    constexpr int kStep = MULTI ? 32 : 16;   // columns at a time
    const int row = threadIdx.x & (kTile - 1);
    const uint32_t lane_base = static_cast<uint32_t>(row & ~31) << 16;
    const int token = row / p.group, head = row - token * p.group;
    Runs list;
    uint32_t n = 0, groups = 0, joined = 0;  // tiles of this stream, groups, groups whose keys are split
    const uint32_t s_addr = tmem + lane_base + s * kTile;
    float* const slots = p.slots + static_cast<int64_t>(blockIdx.x) * p.slots_per_cta * p.slot_floats;
    float M = -INFINITY, L = 0.0f;
    float2 acc[MULTI ? 1 : kHalf / 2];  // the run's sums, unless they stand in slot 0
    Left left{};

    // `n` and `groups` are those behind the group that is left: it is settled before they move on.
    // Its products are complete, non-finite values are in: both warpgroups may read it.
    auto settle = [&]() {
        if (left.tiles) {
            if (!warp_wait(&sh.pv_done[s], (n - 1) & 1u, sh)) return false;
            tmem_fence_after();
            if (left.warp_live &&
                *reinterpret_cast<volatile uint32_t*>(&sh.odd[(groups - 1) % kGroupRing]) == groups)
                add_odd<DP, F16>(p, sh.runs[left.run % kRunRing], left.g, tmem + lane_base + o_column<DP>(groups - 1, s), s);
        }
        if (left.split) {
            tmem_fence_before();
            mbar_arrive(&sh.g_done);
        }
        return true;
    };
    // Joins it and, behind a run's last group, writes what the run has.
    // With `open` the products that wait for O to have been read may then begin.
    auto finish = [&](bool open) {
        left.any = false;
        Join in{0.0f, 1.0f, 0.0f};  // of the group's streams
        float mg = left.mg, lg = left.lg;
        if (left.split) {
            if (!warp_wait(&sh.g_done, joined & 1u, sh)) return false;
            tmem_fence_after();
            in = join_at(sh.ref[0][row], sh.ref[1][row]);
            lg = join_sum(sh.sum[0][row], sh.sum[1][row], in);
            mg = in.m;
        }
        const int col0 = left.split ? s * kHalf : 0;
        const int slot_row = MULTI || !left.split ? s * kTile + row : row;
        const uint32_t at = tmem + lane_base + o_column<DP>(groups - 1, left.split ? 0 : s) + col0;
        const bool write = left.last && left.whole && left.complete && left.live;
        uint16_t* const out = p.out + left.t * p.out_token_stride + left.h * p.out_head_stride + col0;
        Join j{M, 1.0f, 0.0f};
        if (left.whole) {
            j = join_at(M, mg);
            L = join_sum(L, lg, j);
            M = j.m;
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        // the group's kStep columns from `ch` on
        auto load = [&](float2 (&x)[kStep / 2], int ch) {
            uint32_t z[kStep], y[kStep];
            tmem_ld(z, at + ch);
            if (left.both) tmem_ld(y, at + DP + ch);
            tmem_wait_ld(z);
#pragma unroll
            for (int e = 0; e < kStep / 2; ++e) x[e] = make_float2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1]));
            if (left.both) {
                tmem_wait_ld(y);
#pragma unroll
                for (int e = 0; e < kStep / 2; ++e)
                    x[e] = join_sum2(x[e], make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), in);
            }
        };
        auto store = [&](float4* to, const float2* x) {
#pragma unroll
            for (int e = 0; e < kStep / 4; ++e) to[e * p.slot_rows] = make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y);
        };
        auto put = [&](int ch, const float2* x) {
#pragma unroll
            for (int e = 0; e < kStep / 8; ++e) {
                if (col0 + ch + e * 8 >= p.head_dim) break;
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = pack_pair<F16>(x[4 * e + k].x * inv, x[4 * e + k].y * inv);
                *reinterpret_cast<uint4*>(out + ch + e * 8) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        };
        if (MULTI && left.warp_live) {
            // A row's sums would fill 128 registers: they stand in slot 0, for this thread alone, and
            // the next columns are fetched while these are joined.
            float4* const sums = reinterpret_cast<float4*>(slots + (left.whole ? 0 : left.slot * p.slot_floats)) + slot_row;
            const bool join = left.whole && left.g > 0 && left.live;
            const int cols = left.split ? kHalf : DP;
            float4 ahead[kStep / 4];
            auto fetch = [&](int ch) {
#pragma unroll
                for (int e = 0; e < kStep / 4; ++e) ahead[e] = sums[(ch / 4 + e) * p.slot_rows];
            };
            if (join) fetch(0);
#pragma unroll 1
            for (int ch = 0; ch < cols; ch += kStep) {
                float2 x[kStep / 2];
                load(x, ch);
                if (open && ch + kStep >= cols) {
                    tmem_fence_before();
                    mbar_arrive(&sh.p_full[s]);
                }
                if (left.whole) {
#pragma unroll
                    for (int e = 0; e < kStep / 4; ++e) {
                        const float4 a = join ? ahead[e] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        x[2 * e] = join_sum2(make_float2(a.x, a.y), x[2 * e], j);
                        x[2 * e + 1] = join_sum2(make_float2(a.z, a.w), x[2 * e + 1], j);
                    }
                    if (join && ch + kStep < cols) fetch(ch + kStep);
                }
                if (write)
                    put(ch, x);
                else if (left.live)
                    store(sums + ch / 4 * p.slot_rows, x);
            }
        }
        if (MULTI && open && !left.warp_live) {
            tmem_fence_before();
            mbar_arrive(&sh.p_full[s]);
        }
        if (!MULTI && left.warp_live) {
#pragma unroll
            for (int ch = 0; ch < kHalf; ch += kStep) {
                float2 x[kStep / 2];
                load(x, ch);
                if (left.whole) {
#pragma unroll
                    for (int e = 0; e < kStep / 2; ++e) acc[ch / 2 + e] = join_sum2(acc[ch / 2 + e], x[e], j);
                } else if (left.live) {
                    store(reinterpret_cast<float4*>(slots + left.slot * p.slot_floats) + (col0 + ch) / 4 * p.slot_rows + slot_row, x);
                }
            }
        }
        if (left.split) {
            tmem_fence_before();
            mbar_arrive(&sh.o_free[joined & 1u]);
            ++joined;
        }
        if (left.live && !write && (!left.whole || left.last)) {  // joined elsewhere
            float* const slot = slots + (left.whole ? 0 : left.slot * p.slot_floats);
            if (!MULTI && left.whole) {
#pragma unroll
                for (int ch = 0; ch < kHalf; ch += kStep)
                    store(reinterpret_cast<float4*>(slot) + (col0 + ch) / 4 * p.slot_rows + slot_row, acc + ch / 2);
            }
            if (col0 == 0) {
                slot[DP * p.slot_rows + slot_row] = left.whole ? M : mg;
                slot[(DP + 1) * p.slot_rows + slot_row] = left.whole ? L : lg;
            }
        }
        if (write) {
            if (!MULTI) {
#pragma unroll
                for (int ch = 0; ch < kHalf; ch += kStep) put(ch, acc + ch / 2);
            }
            if (col0 == 0 && p.lse != nullptr)
                p.lse[static_cast<int64_t>(left.t) * p.kv_heads * p.group + left.h] = final_lse(M, L);
        }
        if (left.last) {  // the next run starts from nothing
            list.give_back(sh, left.run);
            M = -INFINITY;
            L = 0.0f;
#pragma unroll
            for (int e = 0; e < (MULTI ? 0 : kHalf / 2); ++e) acc[e] = make_float2(0.0f, 0.0f);
        }
        return true;
    };
#pragma unroll
    for (int e = 0; e < (MULTI ? 0 : kHalf / 2); ++e) acc[e] = make_float2(0.0f, 0.0f);

    // Every turn of the inner loop has at most one tile of this stream and what is left of the group
    // before; turns without a tile (no second row tile, a group's only tile is the other stream's, an
    // item without keys, no run is left) have only that.
    for (bool more = true; more; ++list.k) {
        const Run* const next = list.get(sh);
        if (next == nullptr) return;
        const Run& u = *next;
        more = u.r >= 0;
        const bool split = !MULTI || u.split;
        bool idle = !more || (!split && s == 1 && !u.second);
        const int32_t tile = u.tile + (split ? 0 : s);
        const int32_t i = tile * p.tile_tokens + token;
        const bool live = !idle && row < p.tile_tokens * p.group && i < u.na;
        const bool warp_live = __any_sync(0xFFFFFFFFu, live);
        const int32_t mine = live ? i : 0;
        const uint32_t* words = p.mask == nullptr ? nullptr : p.mask + static_cast<int64_t>(u.tok0 + mine) * p.mask_words;
        const int32_t all = seen_by_all(p, u, tile);
        if (!idle && u.nt == 0) {  // no key: nothing is joined, the row is 0
            if (live) {
                const int64_t t_out = u.tok0 + i;
                const int h_out = u.head * p.group + head, col0 = split ? s * kHalf : 0;
                uint16_t* const out = p.out + t_out * p.out_token_stride + h_out * p.out_head_stride + col0;
                for (int e = 0; e < (split ? kHalf : DP) / 8; ++e)
                    if (col0 + e * 8 < p.head_dim) *reinterpret_cast<uint4*>(out + e * 8) = make_uint4(0, 0, 0, 0);
                if (col0 == 0 && p.lse != nullptr) p.lse[t_out * p.kv_heads * p.group + h_out] = -INFINITY;
            }
            // A turn without a tile, as what is left may not wait for scores here: the run that it
            // belongs to keeps its place in the list, and with a few runs like this one behind it the
            // next one that has scores would find no place.
            idle = true;
        }

        const int32_t g1 = idle ? u.ga + 1 : u.gb;
        for (int32_t g = u.ga; g < g1; ++g) {
            const int32_t ta = g * u.gt, tb = idle ? ta : min(ta + u.gt, u.nt);
            const int32_t mine0 = ta + (split ? s : 0);
            const uint32_t column = o_column<DP>(groups, 0);
            RowState st{-INFINITY, 0.0f, 0.0f};
            for (int32_t t = mine0; t == mine0 || t < tb; t += split ? 2 : 1) {
                const bool has = t < tb;
                if (has) {
                    if (!warp_wait(&sh.s_full[s], n & 1u, sh)) return;
                    tmem_fence_after();
                    if (warp_live && !softmax_tile<DP, F16>(p, sh, u, s, s_addr, tmem + lane_base + column + s * DP, t,
                                                            t == mine0, n, all, live, mine, words, st))
                        return;
                }
                const bool due = left.any;
                // a barrier's phase is waited for before the next one can complete
                if (due && !settle()) return;
                // where there is one O, this stream's next products may begin when the group before has
                // been read, unless the other warpgroup reads it too and both say so
                const bool late = due && !left.split && kSums<DP> == 1;
                if (has && !late) {
                    tmem_fence_before();
                    mbar_arrive(&sh.p_full[s]);
                }
                if (due && !finish(MULTI && has && late)) return;
                n += has;
            }
            if (idle) break;
            left.any = true;
            left.split = split;
            left.both = split && ta + 1 < tb;
            left.tiles = mine0 < tb;
            left.live = live;
            left.warp_live = warp_live;
            left.whole = u.ga == 0;  // from the first group on: joined here
            left.last = g + 1 == u.gb;
            left.complete = u.gb == u.ng;
            left.run = list.k;
            left.g = g;
            left.slot = 1 + g - u.ga;
            left.t = u.tok0 + i;
            left.h = u.head * p.group + head;
            left.mg = st.ref == -INFINITY ? -INFINITY : st.off;
            left.lg = st.l;
            if (split) {
                // the other warpgroup has read what stands there
                if (joined > 0 && !warp_wait(&sh.o_free[(joined - 1) & 1u], ((joined - 1) >> 1) & 1u, sh)) return;
                sh.ref[s][row] = left.mg;
                sh.sum[s][row] = left.lg;
            }
            ++groups;
        }
        if (idle && more) {
            if (u.nt > 0) groups += u.gb - u.ga;
            list.give_back(sh, list.k);
        }
    }
}

// Shared memory: Q of two runs, the ring, the barriers.  A product reads 128 rows of Q
// where fewer were copied; what lies behind them gives rows of S that nobody uses.
__host__ __device__ inline size_t attn_shared_bytes(int dp, int stages, int q_chunk)
{
    return static_cast<size_t>(2 * (dp / 64)) * q_chunk + static_cast<size_t>(stages) * kTile * dp * 2 +
           sizeof(Shared);
}

// MULTI: some request may have more rows than one tile.
// The 384 threads launch with 168 registers each; the softmax warps take 208 and the other
// four warps keep 88 (256 * 208 + 128 * 88 = 384 * 168).  Nothing may spill: local memory has
// 25 KB of L1 left beside the ring and costs a trip to L2 for most.
template <int DP, bool F16, bool MULTI>
__global__ void __launch_bounds__(kAttnThreads, 1)
    tree_attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    extern __shared__ __align__(1024) unsigned char base[];  // the swizzle repeats every 1024 bytes
    unsigned char* ring = base + 2 * (DP / 64) * p.q_chunk;
    Shared& sh = *reinterpret_cast<Shared*>(ring + static_cast<size_t>(p.stages) * (kTile * DP * 2));
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_launch_dependents();
    Lengths mine{};
    if (tid < p.R) mine = lengths_of(p, tid);  // on their way while the barriers are made
    if ((smem_addr(base) & 1023u) != 0) {  // never seen: the array's alignment is declared
        if (tid == 0) p.flags[blockIdx.x] = kFlagTimeout;
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 2);  // its products, and warp 3
            mbar_init(&sh.v_ok[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], kTile);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.g_done, 2 * kTile);
        mbar_init(&sh.o_free[0], 2 * kTile);
        mbar_init(&sh.o_free[1], 2 * kTile);
        for (int i = 0; i < kRunRing; ++i) {
            mbar_init(&sh.run_full[i], 1);
            mbar_init(&sh.run_empty[i], kRunReaders);
        }
        mbar_init(&sh.drain, 1);
        fence_barrier_init();
        sh.stop = static_cast<int32_t>(blockIdx.x) == p.stop_cta ? 1 : 0;
    }
    if (tid < kGroupRing) sh.odd[tid] = 0;
    if (warp == 2) tmem_alloc(&sh.tmem, 512);
    tmem_fence_before();
    find_share(p, sh, mine);  // ends with a barrier
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    if (tid == 0) {
        p.starts[blockIdx.x] = sh.start;
        p.firsts[blockIdx.x] = sh.first;
        if (blockIdx.x + 1 == gridDim.x) p.starts[gridDim.x] = Start{p.R, 0, 0, 0};
    }

    if (warp < 4) {
        registers_lower<88>();
        if (warp == 0)
            copy_tiles<DP>(p, sh, ring, &mk, 0);
        else if (warp == 1)
            issue_products<DP, MULTI>(p, sh, smem_addr(base), smem_addr(ring), tmem);
        else if (warp == 2)
            copy_tiles<DP>(p, sh, ring, &mv, 1);
        else
            copy_q_clean_v<DP, F16, MULTI>(p, sh, base, ring, &mq);
    } else {
        registers_raise<208>();
        softmax_rows<DP, F16, MULTI>(p, sh, tmem, (warp - 4) >> 2);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
    if (tid == 0) p.flags[blockIdx.x] = sh.stop != 0 ? kFlagTimeout : 0u;
}

// ---- groups that were cut across CTAs -----------------------------------------------------------
constexpr int kJoinThreads = 256, kAhead = 4, kJoinBlocks = 8;

// A CTA gave up a wait: NaN in every row, so that no caller takes what stands there for results.
__device__ __noinline__ void spoil_rows(const AttnParams& p)
{
    const int32_t heads = p.kv_heads * p.group, vecs = p.head_dim / 8;
    const uint32_t nan = 0x7FFF7FFFu;  // in bf16 as in fp16
    for (int32_t r = blockIdx.y * gridDim.x + blockIdx.x; r < p.R; r += gridDim.x * gridDim.y) {
        const Request q = request_of(p, r);
        const int64_t n = static_cast<int64_t>(q.na) * heads * vecs;
        for (int64_t x = threadIdx.x; x < n; x += kJoinThreads) {
            const int64_t row = x / vecs, t = q.tok0 + row / heads;
            const int32_t v = static_cast<int32_t>(x - row * vecs), h = static_cast<int32_t>(row % heads);
            *reinterpret_cast<uint4*>(p.out + t * p.out_token_stride + h * p.out_head_stride + v * 8) =
                make_uint4(nan, nan, nan, nan);
            if (v == 0 && p.lse != nullptr) p.lse[t * heads + h] = NAN;
        }
    }
}

// blockIdx.x = c: the item that is cut where CTA c's share ends, if its first group lies in that
// share; blockIdx.y: a part of its (row, eight columns).  Groups are joined as softmax_rows does.
// Its time is that of a few dependent loads: eight blocks at most for an item, three on an SM,
// each thread with eight columns (four columns and a block for every 256 of them: 30 us behind
// the attention of 64 x 65 tokens instead of 13).
template <int DP, bool F16>
__global__ void __launch_bounds__(kJoinThreads, 3) attn_join_kernel(const __grid_constant__ AttnParams p, int32_t ctas)
{
    pdl_wait_primary();
    // all shares at once: the ones that an item goes through are read one after the other
    extern __shared__ Start s_starts[];
    const int32_t c = blockIdx.x;
    const Request q = p.firsts[min(c + 1, ctas - 1)];
    uint32_t f = 0;
    for (int32_t i = threadIdx.x; i < ctas; i += kJoinThreads) f |= p.flags[i];
    for (int32_t i = threadIdx.x; i <= ctas; i += kJoinThreads) s_starts[i] = p.starts[i];
    const bool gave_up = __syncthreads_or(static_cast<int>(f)) != 0;
    if (p.status != nullptr && blockIdx.y == 0) {
        for (int32_t r = blockIdx.x * kJoinThreads + threadIdx.x; r < p.R; r += gridDim.x * kJoinThreads)
            p.status[r] = gave_up ? SV_ST_TIMEOUT : 0;
    }
    if (gave_up) {
        spoil_rows(p);
        return;
    }
    const Start s = s_starts[c], e = s_starts[c + 1];
    if (e.g == 0 || (s.r == e.r && s.item == e.item && s.g > 0)) return;
    const int32_t head = e.item / q.per_head, tile0 = 2 * (e.item - head * q.per_head);
    int32_t kv_end;
    const int32_t nt = item_tiles(p, q, tile0, &kv_end);
    const int32_t ng = max(1, (nt + q.gt - 1) / q.gt);
    if (e.g >= ng) return;  // its groups all lie in CTA c's share

    const int64_t at_m0 = static_cast<int64_t>(DP) * p.slot_rows;
    for (int32_t index = blockIdx.y * kJoinThreads + threadIdx.x; index < p.slot_rows * (DP / 8); index += gridDim.y * kJoinThreads) {
        const int32_t slot_row = index % p.slot_rows, c8 = index / p.slot_rows;
        const int32_t tile = tile0 + slot_row / kTile, row = slot_row % kTile;
        const int32_t token = row / p.group, i = tile * p.tile_tokens + token;
        if (c8 * 8 >= p.head_dim || row >= p.tile_tokens * p.group || i >= q.na) continue;

        // where the streams split the keys next to two row tiles' room, the second half of the
        // columns stands in the second tile's rows
        const bool beside = p.slot_rows > kTile && q.tiles == 1 && c8 >= DP / 16;
        const int64_t at_o = (static_cast<int64_t>(beside ? c8 - DP / 16 : c8) * 2 * p.slot_rows + slot_row + (beside ? kTile : 0)) * 4;
        const int64_t at_p = at_o + p.slot_rows * 4, at_m = at_m0 + slot_row, at_l = at_m + p.slot_rows;
        const float* x = p.slots + static_cast<int64_t>(c) * p.slots_per_cta * p.slot_floats;
        float4 sum[2] = {*reinterpret_cast<const float4*>(x + at_o), *reinterpret_cast<const float4*>(x + at_p)};
        float M = x[at_m], L = x[at_l];
        // the other groups, kAhead loaded before the first of them is joined
        int32_t g = e.g, o = c, gb = e.g;
        while (g < ng) {
            float4 y[kAhead][2];
            float mg[kAhead], lg[kAhead];
            int32_t n = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                while (g + n < ng && g + n >= gb) {  // the CTA that has the next group
                    ++o;
                    const Start f = s_starts[o + 1];
                    gb = f.r == e.r && f.item == e.item ? min(ng, f.g) : ng;
                    x = p.slots + (static_cast<int64_t>(o) * p.slots_per_cta + 1) * p.slot_floats;
                }
                if (g + n < ng) {
                    y[k][0] = *reinterpret_cast<const float4*>(x + at_o);
                    y[k][1] = *reinterpret_cast<const float4*>(x + at_p);
                    mg[k] = x[at_m];
                    lg[k] = x[at_l];
                    x += p.slot_floats;
                    ++n;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (k < n) {
                    const Join j = join_at(M, mg[k]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        sum[h].x = join_sum(sum[h].x, y[k][h].x, j);
                        sum[h].y = join_sum(sum[h].y, y[k][h].y, j);
                        sum[h].z = join_sum(sum[h].z, y[k][h].z, j);
                        sum[h].w = join_sum(sum[h].w, y[k][h].w, j);
                    }
                    L = join_sum(L, lg[k], j);
                    M = j.m;
                }
            }
            g += n;
        }
        const int64_t t = q.tok0 + i;
        const int32_t h = head * p.group + (row - token * p.group);
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        uint4 v;
        v.x = pack_pair<F16>(sum[0].x * inv, sum[0].y * inv);
        v.y = pack_pair<F16>(sum[0].z * inv, sum[0].w * inv);
        v.z = pack_pair<F16>(sum[1].x * inv, sum[1].y * inv);
        v.w = pack_pair<F16>(sum[1].z * inv, sum[1].w * inv);
        *reinterpret_cast<uint4*>(p.out + t * p.out_token_stride + h * p.out_head_stride + c8 * 8) = v;
        if (c8 == 0 && p.lse != nullptr) p.lse[t * p.kv_heads * p.group + h] = final_lse(M, L);
    }
}

// ---- host ------------------------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

bool encode(CUtensorMap* map, int dtype, int rank, const void* data, const uint64_t* dims, const int64_t* strides,
            const uint32_t* box)
{
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    cuuint64_t d[5], st[5];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        // an axis with one step has a stride that is never used; the map wants one above 0 all the same
        if (i > 0) st[i - 1] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i] * 2 : std::max<int64_t>(strides[i] / 8 * 16, 16));
    }
    return fn(map, dtype == SV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              static_cast<cuuint32_t>(rank), const_cast<void*>(data), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int attn_ctas()
{
    const int n = device_sm_count();
    return n > 0 ? n : 152;
}

struct AttnLayout {
    int32_t tile_tokens, slot_rows, slots_per_cta;
    bool multi;  // some request may have more rows than one tile
    int64_t slot_floats;
    size_t starts, firsts, flags, slots, total;
};

// Slots of a CTA: one for the first groups of the item its share ends in, and one for each group of
// the item it begins in.  Those are at most an item's groups, and no more than fit a share (a group
// costs at least 6 on the line, but for an item's last).
AttnLayout attn_layout(int32_t R, int32_t max_tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t max_kv)
{
    AttnLayout a{};
    const int64_t sms = attn_ctas();
    const int32_t G = heads / kv_heads, dp = head_dim <= 64 ? 64 : 128;
    a.tile_tokens = kTile / G;
    const int64_t tiles = (static_cast<int64_t>(max_tokens) + a.tile_tokens - 1) / a.tile_tokens;
    a.multi = tiles > 1;
    a.slot_rows = a.multi ? 2 * kTile : std::min<int32_t>(kTile, (std::max(max_tokens, 1) * G + 7) / 8 * 8);
    a.slot_floats = static_cast<int64_t>(a.slot_rows) * (dp + 2);
    const int64_t nt = (max_kv + kTile - 1) / kTile;
    // Groups of an item, at most (request_of): they are at least 4/5 of the square-root rule's size, and no
    // more than two for every SM that a key head can have.
    const int64_t groups = std::min(2 * std::max<int64_t>(1, sms / kv_heads),
                                    static_cast<int64_t>(1.25 * std::sqrt(static_cast<double>(nt))) + 2);
    const int64_t share = R * std::max<int64_t>(1, (tiles + 1) / 2) * kv_heads * (2 * nt + 2 * groups + 8) / sms + 1;
    a.slots_per_cta = static_cast<int32_t>(1 + std::min(groups, share / 6 + 3));
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    a.starts = 0;
    a.firsts = up(a.starts + static_cast<size_t>(sms + 1) * sizeof(Start));
    a.flags = up(a.firsts + static_cast<size_t>(sms) * sizeof(Request));
    a.slots = up(a.flags + static_cast<size_t>(sms) * 4);
    a.total = up(a.slots + static_cast<size_t>(sms) * a.slots_per_cta * a.slot_floats * 4);
    return a;
}

template <int DP, bool F16, bool MULTI>
cudaError_t launch_attn(const AttnParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                        cudaStream_t stream)
{
    auto kern = tree_attention_kernel<DP, F16, MULTI>;
    const size_t bytes = attn_shared_bytes(DP, p.stages, p.q_chunk);
    // the kernel's shared-memory limit is raised once per device, to the most that it can use
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || ((raised.load(std::memory_order_relaxed) >> dev) & 1u) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxShared));
        if (e != cudaSuccess) return e;
        if (dev < 64) raised.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const int ctas = p.sms;
    kern<<<ctas, kAttnThreads, bytes, stream>>>(p, mq, mk, mv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, std::min(kJoinBlocks, (p.slot_rows * (DP / 8) + kJoinThreads - 1) / kJoinThreads));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(ctas + 1) * sizeof(Start);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<DP, F16>, p, static_cast<int32_t>(ctas));
}

}  // namespace

size_t attn_workspace_bytes(int32_t R, int32_t max_tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
                            int64_t max_kv)
{
    return attn_layout(R, max_tokens, heads, kv_heads, head_dim, max_kv).total;
}

cudaError_t launch_tree_attention(const AttnArgs& a, cudaStream_t stream)
{
    const int32_t max_kv = a.max_blocks * a.cache.block_size;
    const AttnLayout lay = attn_layout(a.R, a.max_tokens, a.q.heads, a.cache.kv_heads, a.q.head_dim, max_kv);
    const bool f16 = a.cache.dtype == SV_F16;
    const int dp = a.q.head_dim <= 64 ? 64 : 128;
    AttnParams p{};
    p.block_table = a.block_table;
    p.kv_len = a.kv_len;
    p.cu_tokens = a.cu_tokens;
    p.mask = a.mask;
    p.R = a.R;
    p.T = a.q.tokens;
    p.max_blocks = a.max_blocks;
    p.max_kv = max_kv;
    p.max_tokens = a.max_tokens;
    p.mask_words = a.mask_words;
    p.by_block = divisor_of(a.cache.block_size);
    p.by_tile = divisor_of(lay.tile_tokens);
    p.block_size = a.cache.block_size;
    p.num_blocks = a.cache.num_blocks;
    p.kv_heads = a.cache.kv_heads;
    p.group = a.q.heads / a.cache.kv_heads;
    p.tile_tokens = lay.tile_tokens;
    p.head_dim = a.q.head_dim;
    p.box_tokens = std::max(1, std::min(lay.tile_tokens, a.max_tokens));
    p.q_chunk = (p.group * p.box_tokens * 128 + 1023) / 1024 * 1024;
    p.box_rows = std::min(kTile, a.cache.block_size & -a.cache.block_size);
    p.sms = attn_ctas();
    p.by_sms = divisor_of(p.sms);
    p.wave = std::max(1, p.sms / p.kv_heads);
    // The ring takes what Q leaves of an SM's 227 KB, in pairs of a stage for K and one for V: 4 or 6 of 32 KB,
    // 12 of 16 KB.  A fifth stage of 32 KB, of which K and V take turns, costs more than it gives: 210.4 us a
    // call for 64 x 65 tokens instead of 205.8, 233.3 for 64 x 32 with 4 heads to a key head instead of 226.0.
    const size_t fixed = attn_shared_bytes(dp, 0, p.q_chunk);
    p.stages = static_cast<int32_t>(std::min<size_t>(kMaxStages, (kMaxShared - fixed) / (kTile * dp * 2))) & ~1;
    // a scale of 0 weighs all alike; the smallest factor keeps hidden scores at -inf
    p.c = std::max(fabsf(a.scale) * 1.44269504088896341f, 1e-30f);
    p.word_qk = product_word(f16, kTile, kTile, false, a.scale < 0.0f);
    p.word_pv = product_word(f16, kTile, static_cast<uint32_t>(dp), true, false);
    p.v = static_cast<const uint16_t*>(a.cache.v);
    p.block_stride = a.cache.block_stride;
    p.token_stride = a.cache.token_stride;
    p.head_stride = a.cache.head_stride;
    p.out = static_cast<uint16_t*>(const_cast<void*>(a.out.data));
    p.out_token_stride = a.out.token_stride;
    p.out_head_stride = a.out.head_stride;
    p.lse = a.lse;
    p.status = a.status;
    char* ws = static_cast<char*>(a.workspace);
    p.starts = reinterpret_cast<Start*>(ws + lay.starts);
    p.firsts = reinterpret_cast<Request*>(ws + lay.firsts);
    p.flags = reinterpret_cast<uint32_t*>(ws + lay.flags);
    p.slots = reinterpret_cast<float*>(ws + lay.slots);
    p.slot_floats = lay.slot_floats;
    p.slots_per_cta = lay.slots_per_cta;
    p.slot_rows = lay.slot_rows;
    p.stop_cta = a.stop_cta;

    CUtensorMap mq, mk, mv;
    const uint64_t D = static_cast<uint64_t>(a.q.head_dim);
    const uint64_t qd[3] = {D, static_cast<uint64_t>(a.q.heads), static_cast<uint64_t>(a.q.tokens)};
    const int64_t qs[3] = {1, a.q.head_stride, a.q.token_stride};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(p.box_tokens)};
    const uint64_t kd[4] = {D, static_cast<uint64_t>(p.block_size), static_cast<uint64_t>(p.kv_heads),
                            static_cast<uint64_t>(p.num_blocks)};
    const int64_t ks[4] = {1, p.token_stride, p.head_stride, p.block_stride};
    const uint32_t kb[4] = {64, static_cast<uint32_t>(p.box_rows), 1, 1};
    if (!encode(&mq, a.cache.dtype, 3, a.q.data, qd, qs, qb) || !encode(&mk, a.cache.dtype, 4, a.cache.k, kd, ks, kb) ||
        !encode(&mv, a.cache.dtype, 4, a.cache.v, kd, ks, kb))
        return cudaErrorInvalidValue;
    const int kind = (dp == 128 ? 4 : 0) | (f16 ? 2 : 0) | (lay.multi ? 1 : 0);
    switch (kind) {
        case 0: return launch_attn<64, false, false>(p, mq, mk, mv, stream);
        case 1: return launch_attn<64, false, true>(p, mq, mk, mv, stream);
        case 2: return launch_attn<64, true, false>(p, mq, mk, mv, stream);
        case 3: return launch_attn<64, true, true>(p, mq, mk, mv, stream);
        case 4: return launch_attn<128, false, false>(p, mq, mk, mv, stream);
        case 5: return launch_attn<128, false, true>(p, mq, mk, mv, stream);
        case 6: return launch_attn<128, true, false>(p, mq, mk, mv, stream);
        default: return launch_attn<128, true, true>(p, mq, mk, mv, stream);
    }
}

}  // namespace sv
