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
//               five stages (the block ids of the next tile are fetched before the
//               wait for a stage);
//   warp 1      issues the products; S in tensor memory, P over S in tensor memory as
//               the left operand of P V, O in tensor memory;
//   warp 3      copies Q, and cleans V where a tile holds positions that not every row sees: rows
//               behind the last key become 0 (P is 0 there, but 0 * NaN is not), and so
//               do NaN and infinite entries, which are noted and added in 32 bits at
//               the end of the group to the rows that do see them;
//   warps 4-7   softmax and sums of the first row tile, one row per thread;
//   warps 8-11  of the second row tile, when requests have more rows than one tile
//               holds: both tiles use the same K and V from shared memory.
//
// Order of sums.  A request's keys are cut into groups of whole tiles by a rule on
// its own lengths (request_of).  Within a group O and the sum l belong to a
// reference m, the row maximum of the group's first tile; a later tile's maximum
// replaces it only when it is more than 2^8 above (O is then rescaled), which no
// 32-bit sum notices.  Groups are joined from the first to the last, (O, l, m) with
// (O', l', m') at max(m, m').  A CTA that has an item from its first group on joins
// in registers; other groups go to the workspace and attn_join_kernel joins them in
// the same order with the same instructions, so the bits do not depend on where the
// work was cut.
//
// Work.  An item is (request, key head, pair of row tiles), a unit one group of an
// item.  All units lie on one line, in cost of tiles plus one per group, cut evenly
// over the CTAs; every CTA finds its share itself from the lengths on the device.
#include <algorithm>
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
constexpr int kMaxStages = 10;
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

struct AttnParams {
    const int32_t *block_table, *kv_len, *cu_tokens;
    const uint32_t* mask;
    int32_t R, T, max_blocks, max_kv, max_tokens, mask_words;
    int32_t block_size, num_blocks, kv_heads, group, tile_tokens, head_dim;
    int32_t pairs;     // row tiles an item holds: 1 or 2
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
    uint32_t* flags;  // [CTAs]
    float* slots;     // [CTAs][slots_per_cta]: O as [DP / 4][rows][4], then m [rows], l [rows]
    int64_t slot_floats;
    int32_t slots_per_cta, slot_rows;
};

struct Request {
    int32_t tok0, na, kv, ctx;  // first token, tokens that attend, keys, keys before the tokens
    int32_t tiles, per_head;    // row tiles; items of a key head
    int32_t gt, ng, cost;       // key tiles of a group, groups and cost of an item over all keys
};

// Groups: one request alone should give about two units to every SM, so the tiles of
// an item are cut into at most 2 * SMs / (key heads * tile pairs) groups; a group
// holds at least 2 tiles (8 where there are more rows than one tile holds: such
// items are bound by the products, and a group's end costs a pass over O).
__device__ __forceinline__ Request request_of(const AttnParams& p, int32_t r)
{
    Request q;
    const int32_t t0 = min(max(p.cu_tokens[r], 0), p.T), t1 = min(max(p.cu_tokens[r + 1], t0), p.T);
    q.tok0 = t0;
    q.na = min(t1 - t0, p.max_tokens);
    q.kv = min(max(p.kv_len[r], 0), p.max_kv);
    q.ctx = q.kv - (t1 - t0);
    q.tiles = (q.na + p.tile_tokens - 1) / p.tile_tokens;
    const int32_t tile_pairs = (q.tiles + 1) / 2;
    q.per_head = p.pairs == 2 ? tile_pairs : q.tiles;
    const int32_t nt = (q.kv + kTile - 1) / kTile;
    const int32_t most = max(1, min(p.sms, 2 * p.sms / max(1, p.kv_heads * tile_pairs)));
    q.gt = max(q.tiles > 1 ? 8 : 2, (nt + most - 1) / most);
    q.ng = max(1, (nt + q.gt - 1) / q.gt);
    q.cost = nt + q.ng;
    return q;
}

// An item's groups that lie in a CTA's share.
struct Run {
    int32_t tok0, na, ctx, kv_end;  // keys [0, kv_end) are looked at
    int32_t head, tile0;            // key head, first row tile
    bool second;                    // a second row tile
    int32_t gt, ga, gb, ng;         // tiles of a group, groups [ga, gb) of ng
    int32_t nt;                     // key tiles of the item
};

struct Walk {
    Start at, end;
    int32_t known;
    Request q;
};

__device__ __forceinline__ int32_t item_tiles(const AttnParams& p, const Request& q, int32_t tile0, int32_t* kv_end)
{
    int32_t e = q.kv;
    if (p.mask == nullptr) e = min(e, q.ctx + min(q.na, (tile0 + p.pairs) * p.tile_tokens));
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
        out.tile0 = (w.at.item - out.head * q.per_head) * p.pairs;
        out.nt = item_tiles(p, q, out.tile0, &out.kv_end);
        out.ng = max(1, (out.nt + q.gt - 1) / q.gt);
        out.ga = w.at.g;
        out.gb = w.end.r == w.at.r && w.end.item == w.at.item ? min(out.ng, w.end.g) : out.ng;
        w.at.item += 1;
        w.at.g = 0;
        if (out.ga >= out.gb) continue;
        out.tok0 = q.tok0;
        out.na = q.na;
        out.ctx = q.ctx;
        out.gt = q.gt;
        out.second = p.pairs == 2 && out.tile0 + 1 < q.tiles;
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
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], drain;
    uint64_t v_ok[kMaxStages];  // the stage's V has been cleaned
    int64_t scan[16];
    Start start, end;
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
// Locate the unit that starts at or behind `at` on the line, inside request r whose
// costs begin at `first`.
__device__ __forceinline__ Start locate(const AttnParams& p, const Request& q, int32_t r, int64_t first, int64_t at)
{
    const int64_t off = at - first;
    int32_t item = static_cast<int32_t>(off / q.cost);
    const int32_t in = static_cast<int32_t>(off - static_cast<int64_t>(item) * q.cost);
    int32_t g = (in + q.gt) / (q.gt + 1);
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

// Every thread of the CTA; sets sh.start and sh.end.
__device__ void find_share(const AttnParams& p, Shared& sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    int64_t mine = 0;
    for (int32_t r = tid; r < p.R; r += nt) mine += request_cost(p, request_of(p, r));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
    if (lane == 0) sh.scan[warp] = mine;
    if (tid == 0) sh.start = sh.end = Start{p.R, 0, 0, 0};
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) total += sh.scan[w];
    const int64_t grid = gridDim.x, c = blockIdx.x;
    const int64_t lo = total * c / grid, hi = total * (c + 1) / grid;
    int64_t base = 0;
    for (int32_t r0 = 0; r0 < p.R; r0 += nt) {
        __syncthreads();
        const int32_t r = r0 + tid;
        Request q{};
        int64_t cost = 0;
        if (r < p.R) {
            q = request_of(p, r);
            cost = request_cost(p, q);
        }
        int64_t sum = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += u;
        }
        if (lane == 31) sh.scan[warp] = sum;
        __syncthreads();
        int64_t first = base + sum - cost;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) first += sh.scan[w];
            base += sh.scan[w];
        }
        if (lo >= first && lo < first + cost) sh.start = locate(p, q, r, first, lo);
        if (hi >= first && hi < first + cost) sh.end = locate(p, q, r, first, hi);
    }
    __syncthreads();
}

// ---- warps 0 and 2: K and V --------------------------------------------------------
// Tile t of the line fills stages 2 t (K) and 2 t + 1 (V) of the ring; warp 0 copies K
// and warp 2 V (one warp for both could not issue the copies of 16-token blocks fast
// enough).  One lane issues, block by block; lane i holds block and place of box i.
template <int DP>
__device__ void copy_tiles(const AttnParams& p, Shared& sh, unsigned char* ring, const CUtensorMap* map, int first)
{
    constexpr int kChunks = DP / 64;
    constexpr uint32_t kStage = kTile * DP * 2;
    const int lane = threadIdx.x & 31;
    Walk w{sh.start, sh.end, -1, {}};
    Run u;
    Ring rt{first, 0};
    int32_t fills = 0;  // of this warp; from the ring's second turn on a stage is waited for
    bool ok = true;
    const int32_t subs = kTile / p.box_rows;
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * 128u;
    while (ok && next_run(p, w, u)) {
        const int32_t* table = p.block_table + static_cast<int64_t>(w.known) * p.max_blocks;
        const int32_t t1 = min(u.gb * u.gt, u.nt);
        int32_t t = u.ga * u.gt;
        if (t >= t1) continue;
        auto block_of = [&](int32_t tile) -> int32_t {
            const int32_t x = tile * kTile + lane * p.box_rows;
            return lane < subs && x < u.kv_end ? table[x / p.block_size] : 0;
        };
        int32_t id = block_of(t);
        for (; t < t1; ++t) {
            const int32_t block = id;
            if (t + 1 < t1) id = block_of(t + 1);  // in flight while this tile is issued
            const int32_t place = (t * kTile + lane * p.box_rows) % p.block_size;
            const int32_t live = min(subs, (u.kv_end - t * kTile + p.box_rows - 1) / p.box_rows);
            uint64_t* full = &sh.kv_full[rt.stage];
            // the stage's fill before this one is the ring's last turn: `first + 2 * fills` stages in
            if (first + 2 * fills >= p.stages && !warp_wait(&sh.kv_empty[rt.stage], rt.phase ^ 1u, sh)) {
                ok = false;
                break;
            }
            unsigned char* dst = ring + static_cast<size_t>(rt.stage) * kStage;
            if (elect_one()) mbar_arrive_expect_tx(full, static_cast<uint32_t>(live) * box_bytes * kChunks);
            for (int sub = 0; sub < live; ++sub) {
                const int32_t blk = __shfl_sync(0xFFFFFFFFu, block, sub), pl = __shfl_sync(0xFFFFFFFFu, place, sub);
                if (elect_one()) {
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch)
                        tma_load_4d(dst + sub * box_bytes + ch * kTile * 128, map, full, ch * 64, pl, u.head, blk);
                }
            }
            __syncwarp();
            ++fills;
            rt.next2(p.stages);
        }
    }
    // a CTA that gave up does not leave before its copies have landed
    if (!ok || sh.stop != 0) {
        for (int32_t i = min(fills, p.stages); i > 0; --i) {
            rt.prev2(p.stages);
            mbar_wait_bounded(&sh.kv_full[rt.stage], rt.phase);
        }
    }
}

// ---- warp 3: Q, and V that not every row sees ---------------------------------------
// Q of a run is copied when the run's first tile is waited for.  The warp follows every stage, also those it has nothing to do with, and each stage waits for
// its arrival before it is filled again: the parity of a barrier tells two fills of a
// stage apart only for a warp that is never a whole turn of the ring ahead or behind.
template <int DP, bool F16>
__device__ void copy_q_clean_v(const AttnParams& p, Shared& sh, unsigned char* q_smem, unsigned char* ring,
                               const CUtensorMap* mq)
{
    constexpr int kChunks = DP / 64;
    constexpr uint32_t kStage = kTile * DP * 2, kQ = kTile * DP * 2;
    constexpr uint32_t kExp = F16 ? 0x7C007C00u : 0x7F807F80u;
    const int lane = threadIdx.x & 31;
    Walk w{sh.start, sh.end, -1, {}};
    Run u;
    Ring rk{0, 0}, rv{1, 0};
    uint32_t group = 0, used[2] = {0, 0};
    int32_t runs = 0;
    const uint32_t q_bytes = static_cast<uint32_t>(p.group * p.tile_tokens * 128 * kChunks);
    auto follow = [&]() {
        const int32_t all = seen_by_all(p, u, u.tile0);
        for (int32_t g = u.ga; g < u.gb; ++g, ++group) {
            const int32_t t1 = min((g + 1) * u.gt, u.nt);
            for (int32_t t = g * u.gt; t < t1; ++t, rk.next2(p.stages), rv.next2(p.stages)) {
                const int32_t x0 = t * kTile;
                if (!warp_wait(&sh.kv_full[rk.stage], rk.phase, sh)) return false;
                if (lane == 0) mbar_arrive(&sh.kv_empty[rk.stage]);
                if (!warp_wait(&sh.kv_full[rv.stage], rv.phase, sh)) return false;
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
                    if (__any_sync(0xFFFFFFFFu, odd) && lane == 0) sh.odd[group % kGroupRing] = group + 1;
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.v_ok[rv.stage]);
                }
                if (lane == 0) mbar_arrive(&sh.kv_empty[rv.stage]);
            }
        }
        return true;
    };
    bool ok = true;
    while (ok && next_run(p, w, u)) {
        if (min(u.gb * u.gt, u.nt) > u.ga * u.gt) {
            const int tiles = u.second ? 2 : 1;
            for (int s = 0; ok && s < tiles; ++s) {
                const int b = p.pairs == 2 ? s : runs & 1;
                if (used[b] > 0) ok = warp_wait(&sh.q_empty[b], (used[b] - 1) & 1u, sh);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sh.q_full[b], q_bytes);
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch)
                        tma_load_3d(q_smem + b * kQ + ch * kTile * 128, mq, &sh.q_full[b], ch * 64, u.head * p.group,
                                    u.tok0 + (u.tile0 + s) * p.tile_tokens);
                }
                __syncwarp();
                ++used[b];
            }
            ++runs;
        }
        ok = ok && follow();
    }
    if (!ok || sh.stop != 0)
        for (int b = 0; b < 2; ++b)
            if (used[b] > 0) mbar_wait_bounded(&sh.q_full[b], (used[b] - 1) & 1u);
}

// ---- warp 1: products -------------------------------------------------------------------
template <int DP>
__device__ void issue_products(const AttnParams& p, Shared& sh, uint32_t q_addr, uint32_t ring_addr, uint32_t tmem)
{
    constexpr uint32_t kStage = kTile * DP * 2, kQ = kTile * DP * 2, kChunk = kTile * 128;
    Walk w{sh.start, sh.end, -1, {}};
    Run u;
    Ring rk{0, 0}, rv{1, 0};  // next key tile to multiply with Q, next value tile
    uint32_t tiles[2] = {0, 0};  // per row tile: PV products issued
    uint32_t q_used[2] = {0, 0};
    uint32_t cleaned = 0;  // a bit per stage: parity of its cleanings
    int32_t runs = 0;

    // S[b] = Q[q] K[stage]
    auto qk = [&](int b, int q, int32_t stage) {
        if (elect_one()) {
            const uint64_t qa = smem_operand(q_addr + q * kQ, 16, 1024);
            const uint64_t kb = smem_operand(ring_addr + stage * kStage, 16, 1024);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const uint32_t off = ((k / 4) * kChunk + (k % 4) * 32) >> 4;
                product_ss(tmem + b * kTile, qa + off, kb + off, p.word_qk, k > 0);
            }
            product_commit(&sh.s_full[b]);
        }
    };
    // O[o] (+)= P[b] V[stage]
    auto pv = [&](int b, int o, int32_t stage, bool add) {
        if (elect_one()) {
            const uint64_t vb = smem_operand(ring_addr + stage * kStage, kChunk, 1024);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                product_ts(tmem + 2 * kTile + o * kTile, tmem + b * kTile + k * 8, vb + ((k * 2048) >> 4), p.word_pv,
                           add || k > 0);
            product_commit(&sh.pv_done[b]);
        }
    };
    auto release = [&](uint64_t* bar) {
        if (elect_one()) product_commit(bar);
    };

    bool ok = true;
    while (ok && next_run(p, w, u)) {
        const int32_t t0 = u.ga * u.gt, t1 = min(u.gb * u.gt, u.nt);
        if (t0 >= t1) continue;
        const int32_t all = seen_by_all(p, u, u.tile0);
        const int rows = u.second ? 2 : 1;
        const int qb = p.pairs == 2 ? 0 : runs & 1;
        for (int s = 0; s < rows; ++s) {
            ok = ok && warp_wait(&sh.q_full[qb + s], q_used[qb + s] & 1u, sh);
            ++q_used[qb + s];
        }
        if (!ok) break;
        tmem_fence_after();
        int32_t in_group = 0;  // tiles of the group so far
        auto wait_v = [&](int32_t t) {
            if (t * kTile + kTile <= all) return warp_wait(&sh.kv_full[rv.stage], rv.phase, sh);
            const bool got = warp_wait(&sh.v_ok[rv.stage], (cleaned >> rv.stage) & 1u, sh);
            cleaned ^= 1u << rv.stage;
            return got;
        };
        if (p.pairs == 1) {
            // one row tile: S alternates between two buffers, Q K^T of the next tile goes ahead of P V
            auto next_qk = [&](int32_t t, uint32_t n) {
                if (!warp_wait(&sh.kv_full[rk.stage], rk.phase, sh)) return false;
                tmem_fence_after();
                qk(n & 1u, qb, rk.stage);
                release(&sh.kv_empty[rk.stage]);
                if (t + 1 == t1) release(&sh.q_empty[qb]);
                rk.next2(p.stages);
                return true;
            };
            ok = next_qk(t0, tiles[0]);
            for (int32_t t = t0; ok && t < t1; ++t) {
                const uint32_t n = tiles[0];
                if (t + 1 < t1) ok = next_qk(t + 1, n + 1);
                ok = ok && wait_v(t) && warp_wait(&sh.p_full[n & 1u], (n >> 1) & 1u, sh);
                if (!ok) break;
                tmem_fence_after();
                pv(n & 1u, 0, rv.stage, in_group > 0);
                release(&sh.kv_empty[rv.stage]);
                rv.next2(p.stages);
                ++tiles[0];
                if (++in_group == u.gt) in_group = 0;
            }
        } else {
            // two row tiles take turns: while one's softmax runs, the other's products do
            ok = warp_wait(&sh.kv_full[rk.stage], rk.phase, sh);
            if (!ok) break;
            tmem_fence_after();
            for (int s = 0; s < rows; ++s) {
                qk(s, s, rk.stage);
                if (t0 + 1 == t1) release(&sh.q_empty[s]);
            }
            release(&sh.kv_empty[rk.stage]);
            rk.next2(p.stages);
            for (int32_t t = t0; ok && t < t1; ++t) {
                for (int s = 0; s < rows; ++s) {
                    ok = ok && warp_wait(&sh.p_full[s], tiles[s] & 1u, sh);
                    if (s == 0) ok = ok && wait_v(t);
                    if (!ok) break;
                    tmem_fence_after();
                    pv(s, s, rv.stage, in_group > 0);
                    ++tiles[s];
                    if (t + 1 < t1) {
                        if (s == 0) {
                            ok = warp_wait(&sh.kv_full[rk.stage], rk.phase, sh);
                            if (!ok) break;
                            tmem_fence_after();
                        }
                        qk(s, s, rk.stage);
                        if (t + 2 == t1) release(&sh.q_empty[s]);
                    }
                }
                if (!ok) break;
                release(&sh.kv_empty[rv.stage]);
                rv.next2(p.stages);
                if (t + 1 < t1) {
                    release(&sh.kv_empty[rk.stage]);
                    rk.next2(p.stages);
                }
                if (++in_group == u.gt) in_group = 0;
            }
        }
        ++runs;
    }
    if (!ok || sh.stop != 0) {  // the products that were issued end before tensor memory is given back
        release(&sh.drain);
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

// 16 probabilities of a row: 2^(c z - m), hidden ones 0; packed over the scores
template <bool F16, bool MASKED>
__device__ __forceinline__ void exp_chunk(const uint32_t (&z)[16], uint32_t bits, float2 c2, float2 off2, float2& s0,
                                          float2& s1, uint32_t addr)
{
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float2 x = fma2(make_float2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])), c2, off2);
        x.x = exp2_fast(x.x);
        x.y = exp2_fast(x.y);
        if (MASKED) {
            x.x = (bits >> (2 * e)) & 1u ? x.x : 0.0f;
            x.y = (bits >> (2 * e + 1)) & 1u ? x.y : 0.0f;
        }
        if (e & 1)
            s1 = add2(s1, x);
        else
            s0 = add2(s0, x);
        pk[e] = pack_pair<F16>(x.x, x.y);
    }
    tmem_st8(addr, pk);
}

// A row's probabilities of a whole tile, and their sum.  The loads of 16 scores run
// while the 16 before them are worked on; P lies over scores that have been read.
template <bool F16, bool MASKED>
__device__ __forceinline__ float exp_tile(uint32_t s_addr, const uint32_t (&bits)[4], float c, float off)
{
    const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
    float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
    uint32_t za[16], zb[16];
    tmem_ld16(za, s_addr);
#pragma unroll
    for (int ch = 0; ch < 8; ch += 2) {
        tmem_wait_ld(za);
        tmem_ld16(zb, s_addr + (ch + 1) * 16);
        exp_chunk<F16, MASKED>(za, bits[ch / 2], c2, off2, s0, s1, s_addr + ch * 8);
        tmem_wait_ld(zb);
        if (ch + 2 < 8) tmem_ld16(za, s_addr + (ch + 2) * 16);
        exp_chunk<F16, MASKED>(zb, bits[ch / 2] >> 16, c2, off2, s0, s1, s_addr + (ch + 1) * 8);
    }
    s0 = add2(s0, s1);
    return s0.x + s0.y;
}

template <int DP, bool F16, int PAIRS>
__device__ void softmax_rows(const AttnParams& p, Shared& sh, uint32_t tmem, int s)
{
    const int row = threadIdx.x & (kTile - 1);
    const uint32_t lane_base = static_cast<uint32_t>(row & ~31) << 16;
    const int D = p.head_dim;
    const float c = p.c;
    const int token = row / p.group, head = row - token * p.group;
    Walk w{sh.start, sh.end, -1, {}};
    Run u;
    uint32_t n = 0, group = 0;  // key tiles and groups so far
    float2 acc[DP / 2];
    // The product of tile x is waited for on the barrier of its S buffer: the buffer's next tile
    // is not there before that product is complete, so the barrier is never a phase behind.
    auto wait_pv = [&](uint32_t x) {
        return PAIRS == 2 ? warp_wait(&sh.pv_done[s], x & 1u, sh) : warp_wait(&sh.pv_done[x & 1u], (x >> 1) & 1u, sh);
    };
    const uint32_t o_addr = tmem + lane_base + 2 * kTile + s * kTile;

    while (next_run(p, w, u)) {
        if (s == 1 && !u.second) {
            group += u.gb - u.ga;
            continue;
        }
        const int32_t i = (u.tile0 + s) * p.tile_tokens + token;
        const bool live = row < p.tile_tokens * p.group && i < u.na;
        const bool warp_live = __any_sync(0xFFFFFFFFu, live);
        const int32_t mine = live ? i : 0;
        const uint32_t* words = p.mask == nullptr ? nullptr : p.mask + static_cast<int64_t>(u.tok0 + mine) * p.mask_words;
        const int32_t all = seen_by_all(p, u, u.tile0 + s), cleaned = seen_by_all(p, u, u.tile0);
        const bool whole = u.ga == 0;  // from the first group on: joined here
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int e = 0; e < DP / 2; ++e) acc[e] = make_float2(0.0f, 0.0f);
        const int32_t slot_row = s * kTile + row;
        float* const slots = p.slots + static_cast<int64_t>(blockIdx.x) * p.slots_per_cta * p.slot_floats;

        for (int32_t g = u.ga; g < u.gb; ++g, ++group) {
            const int32_t ta = g * u.gt, tb = min(ta + u.gt, u.nt);
            float ref = -INFINITY, off = 0.0f, l = 0.0f;
            for (int32_t t = ta; t < tb; ++t, ++n) {
                const int b = PAIRS == 2 ? s : static_cast<int>(n & 1u);
                const uint32_t turn = PAIRS == 2 ? n & 1u : (n >> 1) & 1u;
                if (!warp_wait(&sh.s_full[b], turn, sh)) return;
                tmem_fence_after();
                if (warp_live) {
                    const uint32_t s_addr = tmem + lane_base + b * kTile;
                    const int32_t x0 = t * kTile;
                    const bool masked = x0 + kTile > all;
                    uint32_t bits[4] = {0, 0, 0, 0};
                    float top;
                    if (masked) {
                        top = -INFINITY;
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
                            if (live) bits[ch] = seen_bits(p, u, mine, words, x0 + ch * 32);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t z[16];
                                tmem_ld16(z, s_addr + ch * 32 + half * 16);
                                tmem_wait_ld(z);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    top = fmaxf(top, (bits[ch] >> (half * 16 + e)) & 1u ? __uint_as_float(z[e]) : -INFINITY);
                            }
                        }
                    } else {
                        top = -INFINITY;
#pragma unroll 1
                        for (int col = 0; col < kTile; col += 32) top = fmaxf(top, tmem_max32(s_addr + col));
                    }
                    if (t == ta) {
                        ref = top;
                    } else {
                        const bool grow = live && top > ref && (ref == -INFINITY || (top - ref) * c > kGrow);
                        if (__any_sync(0xFFFFFFFFu, grow)) {
                            float f = 1.0f;
                            if (grow) {
                                f = ref == -INFINITY ? 0.0f : exp2_fast((ref - top) * c);
                                ref = top;
                            }
                            l *= f;
                            if (!wait_pv(n - 1)) return;
                            tmem_fence_after();
#pragma unroll 1
                            for (int ch = 0; ch < DP / 32; ++ch) {
                                uint32_t z[32];
                                tmem_ld32(z, o_addr + ch * 32);
                                tmem_wait_ld(z);
#pragma unroll
                                for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(__uint_as_float(z[e]) * f);
                                tmem_st32(o_addr + ch * 32, z);
                            }
                        }
                    }
                    off = ref == -INFINITY ? 0.0f : ref * c;
                    l += masked ? exp_tile<F16, true>(s_addr, bits, c, off) : exp_tile<F16, false>(s_addr, bits, c, off);
                    tmem_wait_st();
                }
                tmem_fence_before();
                mbar_arrive(&sh.p_full[b]);
            }

            // the group's end: O, l and the reference
            const float mg = ref == -INFINITY ? -INFINITY : off;
            const bool any = tb > ta;
            if (any) {
                if (!wait_pv(n - 1)) return;
                tmem_fence_after();
            }
            if (!warp_live) continue;
            if (any && *reinterpret_cast<volatile uint32_t*>(&sh.odd[group % kGroupRing]) == group + 1) {
                // non-finite values join the sums of the rows that see them
                const int32_t x1 = min(tb * kTile, u.kv_end);
                const int32_t* table = p.block_table + static_cast<int64_t>(w.known) * p.max_blocks;
#pragma unroll 1
                for (int ch = 0; ch < DP / 32; ++ch) {
                    uint32_t z[32];
                    tmem_ld32(z, o_addr + ch * 32);
                    tmem_wait_ld(z);
#pragma unroll 1
                    for (int32_t x = max(ta * kTile, cleaned); live && x < x1; ++x) {
                        if (!(seen_bits(p, u, i, words, x) & 1u)) continue;
                        const int32_t blk = table[x / p.block_size];
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const uint16_t* v = p.v + blk * p.block_stride + (x % p.block_size) * p.token_stride +
                                            u.head * p.head_stride + ch * 32;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (ch * 32 + e < D) {
                                const float y = widen<F16>(v[e]);
                                if (!isfinite(y)) z[e] = __float_as_uint(__uint_as_float(z[e]) + y);
                            }
                        }
                    }
                    __syncwarp();
                    tmem_st32(o_addr + ch * 32, z);
                }
                tmem_wait_st();
            }
            const Join j = join_at(M, mg);
            float* slot = slots + static_cast<int64_t>(1 + g - u.ga) * p.slot_floats;
#pragma unroll
            for (int ch = 0; ch < DP / 16; ++ch) {
                uint32_t z[16];
                if (any) {
                    tmem_ld16(z, o_addr + ch * 16);
                    tmem_wait_ld(z);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = 0u;
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[ch * 8 + e] =
                            join_sum2(acc[ch * 8 + e],
                                      make_float2(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1])), j);
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        reinterpret_cast<uint4*>(slot)[(ch * 4 + e) * p.slot_rows + slot_row] =
                            make_uint4(z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
                }
            }
            if (whole) {
                L = join_sum(L, l, j);
                M = j.m;
            } else if (live) {
                slot[DP * p.slot_rows + slot_row] = mg;
                slot[(DP + 1) * p.slot_rows + slot_row] = l;
            }
        }
        if (!whole || !live) continue;
        if (u.gb == u.ng) {
            const int64_t t = u.tok0 + i;
            const int h = u.head * p.group + head;
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            uint16_t* dst = p.out + t * p.out_token_stride + h * p.out_head_stride;
#pragma unroll
            for (int e = 0; e < DP / 8; ++e) {
                if (e * 8 < D) {
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = pack_pair<F16>(acc[4 * e + k].x * inv, acc[4 * e + k].y * inv);
                    *reinterpret_cast<uint4*>(dst + e * 8) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (p.lse != nullptr) p.lse[t * p.kv_heads * p.group + h] = final_lse(M, L);
        } else {
#pragma unroll
            for (int e = 0; e < DP / 4; ++e)
                reinterpret_cast<float4*>(slots)[e * p.slot_rows + slot_row] =
                    make_float4(acc[2 * e].x, acc[2 * e].y, acc[2 * e + 1].x, acc[2 * e + 1].y);
            slots[DP * p.slot_rows + slot_row] = M;
            slots[(DP + 1) * p.slot_rows + slot_row] = L;
        }
    }
}

constexpr size_t attn_shared_bytes(int dp, int stages)
{
    return 1024 + static_cast<size_t>(2 + stages) * kTile * dp * 2 + sizeof(Shared);
}

template <int DP, bool F16, int PAIRS>
__global__ void __launch_bounds__(PAIRS == 2 ? 384 : 256, 1)
    tree_attention_kernel(const AttnParams p, const __grid_constant__ CUtensorMap mq,
                          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    constexpr uint32_t kQ = kTile * DP * 2;
    unsigned char* ring = base + 2 * kQ;
    Shared& sh = *reinterpret_cast<Shared*>(ring + static_cast<size_t>(p.stages) * kQ);
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_launch_dependents();

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
        mbar_init(&sh.drain, 1);
        fence_barrier_init();
        sh.stop = 0;
    }
    if (tid < kGroupRing) sh.odd[tid] = 0;
    if (warp == 2) tmem_alloc(&sh.tmem, 512);
    tmem_fence_before();
    find_share(p, sh);  // ends with a barrier
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    if (tid == 0) {
        p.starts[blockIdx.x] = sh.start;
        if (blockIdx.x + 1 == gridDim.x) p.starts[gridDim.x] = Start{p.R, 0, 0, 0};
    }

    if (warp < 4) {
        if (warp == 0)
            copy_tiles<DP>(p, sh, ring, &mk, 0);
        else if (warp == 1)
            issue_products<DP>(p, sh, smem_addr(base), smem_addr(ring), tmem);
        else if (warp == 2)
            copy_tiles<DP>(p, sh, ring, &mv, 1);
        else
            copy_q_clean_v<DP, F16>(p, sh, base, ring, &mq);
    } else {
        softmax_rows<DP, F16, PAIRS>(p, sh, tmem, PAIRS == 2 ? (warp - 4) >> 2 : 0);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
    if (tid == 0) p.flags[blockIdx.x] = sh.stop != 0 ? kFlagTimeout : 0u;
}

// ---- groups that were cut across CTAs -----------------------------------------------------------
constexpr int kJoinThreads = 256;

// blockIdx.x = c: the item that is cut where CTA c's share ends, if its first group lies in that
// share; blockIdx.y: 256 of its (row, four columns).  Groups are joined as softmax_rows does.
template <int DP, bool F16>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams p, int32_t ctas)
{
    pdl_wait_primary();
    if (p.status != nullptr && blockIdx.y == 0) {
        uint32_t f = 0;
        for (int32_t i = threadIdx.x; i < ctas; i += kJoinThreads) f |= p.flags[i];
        const int32_t st = __syncthreads_or(static_cast<int>(f)) != 0 ? SV_ST_TIMEOUT : 0;
        for (int32_t r = blockIdx.x * kJoinThreads + threadIdx.x; r < p.R; r += gridDim.x * kJoinThreads)
            p.status[r] = st;
    }
    const int32_t c = blockIdx.x;
    const Start s = p.starts[c], e = p.starts[c + 1];
    if (e.g == 0 || (s.r == e.r && s.item == e.item && s.g > 0)) return;
    const Request q = request_of(p, e.r);
    const int32_t head = e.item / q.per_head, tile0 = (e.item - head * q.per_head) * p.pairs;
    int32_t kv_end;
    const int32_t nt = item_tiles(p, q, tile0, &kv_end);
    const int32_t ng = max(1, (nt + q.gt - 1) / q.gt);
    if (e.g >= ng) return;  // its groups all lie in CTA c's share

    const int32_t index = blockIdx.y * kJoinThreads + threadIdx.x;
    const int32_t slot_row = index % p.slot_rows, c4 = index / p.slot_rows;
    if (c4 * 4 >= p.head_dim) return;
    const int32_t tile = tile0 + slot_row / kTile, row = slot_row % kTile;
    const int32_t token = row / p.group, i = tile * p.tile_tokens + token;
    if (row >= p.tile_tokens * p.group || i >= q.na) return;

    const int64_t at_o = (static_cast<int64_t>(c4) * p.slot_rows + slot_row) * 4;
    const int64_t at_m = static_cast<int64_t>(DP) * p.slot_rows + slot_row, at_l = at_m + p.slot_rows;
    const float* x = p.slots + static_cast<int64_t>(c) * p.slots_per_cta * p.slot_floats;
    float4 acc = *reinterpret_cast<const float4*>(x + at_o);
    float M = x[at_m], L = x[at_l];
    int32_t g = e.g;
    for (int32_t o = c + 1; g < ng; ++o) {
        const Start f = p.starts[o + 1];
        const int32_t gb = f.r == e.r && f.item == e.item ? min(ng, f.g) : ng;
        x = p.slots + (static_cast<int64_t>(o) * p.slots_per_cta + 1) * p.slot_floats;
#pragma unroll 4
        for (; g < gb; ++g, x += p.slot_floats) {
            const float4 y = *reinterpret_cast<const float4*>(x + at_o);
            const float mg = x[at_m], lg = x[at_l];
            const Join j = join_at(M, mg);
            acc.x = join_sum(acc.x, y.x, j);
            acc.y = join_sum(acc.y, y.y, j);
            acc.z = join_sum(acc.z, y.z, j);
            acc.w = join_sum(acc.w, y.w, j);
            L = join_sum(L, lg, j);
            M = j.m;
        }
    }
    const int64_t t = q.tok0 + i;
    const int32_t h = head * p.group + (row - token * p.group);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint2 v;
    v.x = pack_pair<F16>(acc.x * inv, acc.y * inv);
    v.y = pack_pair<F16>(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + t * p.out_token_stride + h * p.out_head_stride + c4 * 4) = v;
    if (c4 == 0 && p.lse != nullptr) p.lse[t * p.kv_heads * p.group + h] = final_lse(M, L);
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
    int32_t pairs, tile_tokens, slot_rows, slots_per_cta;
    int64_t slot_floats;
    size_t starts, flags, slots, total;
};

// Slots of a CTA: one for the first groups of the item its share ends in, and one for each group of
// the item it begins in.  Those are at most an item's groups, and no more than fit a share (a group
// costs at least 3 on the line, but for an item's last).
AttnLayout attn_layout(int32_t R, int32_t max_tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t max_kv)
{
    AttnLayout a{};
    const int64_t sms = attn_ctas();
    const int32_t G = heads / kv_heads, dp = head_dim <= 64 ? 64 : 128;
    a.tile_tokens = kTile / G;
    const int64_t tiles = (static_cast<int64_t>(max_tokens) + a.tile_tokens - 1) / a.tile_tokens;
    a.pairs = tiles > 1 ? 2 : 1;
    a.slot_rows = a.pairs == 2 ? 2 * kTile : std::min<int32_t>(kTile, (std::max(max_tokens, 1) * G + 7) / 8 * 8);
    a.slot_floats = static_cast<int64_t>(a.slot_rows) * (dp + 2);
    const int64_t nt = (max_kv + kTile - 1) / kTile;
    const int64_t groups = std::max<int64_t>(1, std::min(std::max<int64_t>(1, std::min(sms, 2 * sms / kv_heads)), (nt + 1) / 2));
    const int64_t share = R * std::max<int64_t>(1, (tiles + 1) / 2) * kv_heads * (nt + groups) / sms + 1;
    a.slots_per_cta = static_cast<int32_t>(1 + std::min(groups, share / 3 + 3));
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    a.starts = 0;
    a.flags = up(a.starts + static_cast<size_t>(sms + 1) * sizeof(Start));
    a.slots = up(a.flags + static_cast<size_t>(sms) * 4);
    a.total = up(a.slots + static_cast<size_t>(sms) * a.slots_per_cta * a.slot_floats * 4);
    return a;
}

template <int DP, bool F16, int PAIRS>
cudaError_t launch_attn(const AttnParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                        cudaStream_t stream)
{
    auto kern = tree_attention_kernel<DP, F16, PAIRS>;
    const size_t bytes = attn_shared_bytes(DP, p.stages);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
    const int ctas = attn_ctas();
    kern<<<ctas, PAIRS == 2 ? 384 : 256, bytes, stream>>>(p, mq, mk, mv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas, (p.slot_rows * (DP / 4) + kJoinThreads - 1) / kJoinThreads);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<DP, F16>, p, static_cast<int32_t>(ctas));
}

}  // namespace

size_t attn_workspace_bytes(int32_t R, int32_t, int32_t max_tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
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
    p.block_size = a.cache.block_size;
    p.num_blocks = a.cache.num_blocks;
    p.kv_heads = a.cache.kv_heads;
    p.group = a.q.heads / a.cache.kv_heads;
    p.tile_tokens = lay.tile_tokens;
    p.head_dim = a.q.head_dim;
    p.pairs = lay.pairs;
    p.box_rows = std::min(kTile, a.cache.block_size & -a.cache.block_size);
    p.sms = attn_ctas();
    p.stages = dp == 128 ? 5 : 10;
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
    p.flags = reinterpret_cast<uint32_t*>(ws + lay.flags);
    p.slots = reinterpret_cast<float*>(ws + lay.slots);
    p.slot_floats = lay.slot_floats;
    p.slots_per_cta = lay.slots_per_cta;
    p.slot_rows = lay.slot_rows;

    CUtensorMap mq, mk, mv;
    const uint64_t D = static_cast<uint64_t>(a.q.head_dim);
    const uint64_t qd[3] = {D, static_cast<uint64_t>(a.q.heads), static_cast<uint64_t>(a.q.tokens)};
    const int64_t qs[3] = {1, a.q.head_stride, a.q.token_stride};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(p.tile_tokens)};
    const uint64_t kd[4] = {D, static_cast<uint64_t>(p.block_size), static_cast<uint64_t>(p.kv_heads),
                            static_cast<uint64_t>(p.num_blocks)};
    const int64_t ks[4] = {1, p.token_stride, p.head_stride, p.block_stride};
    const uint32_t kb[4] = {64, static_cast<uint32_t>(p.box_rows), 1, 1};
    if (!encode(&mq, a.cache.dtype, 3, a.q.data, qd, qs, qb) || !encode(&mk, a.cache.dtype, 4, a.cache.k, kd, ks, kb) ||
        !encode(&mv, a.cache.dtype, 4, a.cache.v, kd, ks, kb))
        return cudaErrorInvalidValue;
    const int kind = (dp == 128 ? 4 : 0) | (f16 ? 2 : 0) | (p.pairs == 2 ? 1 : 0);
    switch (kind) {
        case 0: return launch_attn<64, false, 1>(p, mq, mk, mv, stream);
        case 1: return launch_attn<64, false, 2>(p, mq, mk, mv, stream);
        case 2: return launch_attn<64, true, 1>(p, mq, mk, mv, stream);
        case 3: return launch_attn<64, true, 2>(p, mq, mk, mv, stream);
        case 4: return launch_attn<128, false, 1>(p, mq, mk, mv, stream);
        case 5: return launch_attn<128, false, 2>(p, mq, mk, mv, stream);
        case 6: return launch_attn<128, true, 1>(p, mq, mk, mv, stream);
        default: return launch_attn<128, true, 2>(p, mq, mk, mv, stream);
    }
}

}  // namespace sv
