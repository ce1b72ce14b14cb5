// Pages of the cache: sv_cache_fork, sv_cache_free and sv_cache_compact.
//
// Who holds a block is read from the tables each time: sets of blocks are bit maps in the
// shared memory of one cluster, whose CTAs read the tables together, join their maps, and
// take prefix sums over the bits for an order that does not depend on the threads'.  What moves data (a fork's last blocks, a compaction)
// runs over the whole GPU.
#include <algorithm>
#include <cooperative_groups.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kForkThreads = 128;
constexpr int kMoveBatch = 8;

// ---- fork -------------------------------------------------------------------
// What row r asks for.
struct Fork {
    int32_t source, tokens;  // tokens of the source
    uint32_t bad;
    bool makes, needs;       // a fork, and one that needs a block
};

__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int32_t r)
{
    Fork f{a.source[r], 0, 0u, false, false};
    const int32_t own = a.seq_len[r];
    const int64_t room = static_cast<int64_t>(a.max_blocks) * a.cache.block_size;
    if (own < 0 || own > room) f.bad |= SV_ST_BAD_LENGTH;
    if (f.source < 0) return f;
    if (f.source >= a.R || own != 0) {
        f.bad |= SV_ST_BAD_SOURCE;
        return f;
    }
    f.tokens = a.seq_len[f.source];
    if (f.tokens < 0 || f.tokens > room) {
        f.bad |= SV_ST_BAD_LENGTH;
        return f;
    }
    f.makes = true;
    f.needs = f.tokens - a.by_block.quotient(f.tokens) * a.cache.block_size > 0;
    return f;
}

// Grid: x = rows, y = 128 16-byte columns of the heads of all layers, K and V, z = shares of the tokens.  A
// thread owns a column and walks its share of the source's last block, eight loads before their stores.
// Bound by bytes behind a chain of loads (source, length, blocks taken before, block ids), of which the first
// loads wait for no more than the source's: 23.0 us for 64 forks of 16 layers, 134 MB, 5.8 TB/s, 0.86 of a copy's rate
// (25.1 with one share, 23.9 with loads behind the chain); 3.6 us for 7 forks of 4 layers.
__global__ void __launch_bounds__(kForkThreads) cache_fork_kernel(const ForkArgs a)
{
    const int tid = threadIdx.x;
    const int32_t r = blockIdx.x;
    const bool first = blockIdx.y == 0 && blockIdx.z == 0, teller = r + 1 == a.R && first;  // it tells how many blocks are left
    const Fork f = fork_of(a, r);
    const int32_t full = a.by_block.quotient(max(f.tokens, 0)), tail = f.tokens - full * a.cache.block_size;
    if (!first && (!f.needs || static_cast<int64_t>(blockIdx.z) * kMoveBatch >= tail)) return;
    const int32_t N = a.cache.num_blocks, given = a.free_count[0];
    const int32_t* from = a.block_table + static_cast<int64_t>(f.makes ? f.source : 0) * a.max_blocks;
    const int32_t last = f.needs ? from[full] : -1;

    // the first tokens are on their way while the block they go to is found
    const int32_t vecs = a.cache.head_dim / 8, columns = a.cache.kv_heads * vecs;
    const int64_t column = static_cast<int64_t>(blockIdx.y) * kForkThreads + tid;
    const int32_t plane = static_cast<int32_t>(column / columns),
                  col = static_cast<int32_t>(column - static_cast<int64_t>(plane) * columns), h = col / vecs;
    const bool moves = f.needs && last >= 0 && last < N && plane < 2 * a.cache.layers;
    uint16_t* p = static_cast<uint16_t*>((plane & 1) ? a.cache.v : a.cache.k) + (plane >> 1) * a.cache.layer_stride +
                  h * a.cache.head_stride + (col - h * vecs) * 8;
    const uint16_t* src = p + last * a.cache.block_stride;
    uint4 val[kMoveBatch];
    auto load = [&](int32_t i0) {
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (i0 + u < tail) val[u] = *reinterpret_cast<const uint4*>(src + (i0 + u) * a.cache.token_stride);
    };
    int32_t i0 = blockIdx.z * kMoveBatch;
    if (moves) load(i0);

    int32_t before = 0;  // blocks taken by the rows before
    if (f.needs || teller) {
        for (int32_t i = tid; i < r; i += kForkThreads) before += fork_of(a, i).needs;
        __shared__ int32_t s_sum[kForkThreads / 32];
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        if ((tid & 31) == 0) s_sum[tid >> 5] = before;
        __syncthreads();
        before = 0;
#pragma unroll
        for (int i = 0; i < kForkThreads / 32; ++i) before += s_sum[i];
    }
    const int32_t count = min(max(given, 0), N);
    const bool takes = f.needs && before < count;
    const int32_t fresh = takes ? a.free_blocks[count - 1 - before] : -1;
    const bool done = f.makes && (takes || !f.needs);
    if (first) {
        bool out = takes && (fresh < 0 || fresh >= N || last < 0 || last >= N);
        if (done) {
            int32_t* to = a.block_table + static_cast<int64_t>(r) * a.max_blocks;
            for (int32_t i = tid; i < full; i += kForkThreads) {
                const int32_t id = from[i];
                out = out || id < 0 || id >= N;
                to[i] = id;
            }
            if (takes && tid == 0) to[full] = fresh;
        }
        out = __syncthreads_or(out);
        if (tid == 0) {
            a.seq_len_out[r] = done ? f.tokens : a.seq_len[r];
            if (a.status != nullptr)
                a.status[r] = static_cast<int32_t>(f.bad | (f.makes && !done ? SV_ST_NO_BLOCKS : 0u) |
                                                   (out ? SV_ST_BAD_BLOCK : 0u));
            if (teller) a.free_count_out[0] = max(count - before - (f.needs ? 1 : 0), 0);
        }
    }
    // a stack that holds the source's own block leaves it as it is
    if (!takes || !moves || fresh < 0 || fresh >= N || fresh == last) return;
    uint16_t* dst = p + fresh * a.cache.block_stride;
    while (true) {
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (i0 + u < tail) *reinterpret_cast<uint4*>(dst + (i0 + u) * a.cache.token_stride) = val[u];
        i0 += gridDim.z * kMoveBatch;
        if (i0 >= tail) break;
        load(i0);
    }
}

// ---- sets of blocks over a cluster --------------------------------------------
constexpr int kSetThreads = 1024;
constexpr int kSetCtas = 16;
constexpr int kSetWarps = kSetCtas * kSetThreads / 32;
constexpr int kSetBatch = 8;                 // entries that a thread loads before it sets their bits
constexpr int kSetOwnBytes = 200 * 1024;     // largest bit maps of which every CTA has one of its own
static_assert(kSetOwnBytes <= kMostShared && 2 * (SV_MAX_BLOCKS / 8 / kSetCtas) <= kMostShared, "the largest pool's maps must fit");

// The words of a bit map over [0, num_blocks) are shared out among the CTAs in equal parts.
__host__ __device__ inline int32_t set_words(int32_t num_blocks)
{
    const int32_t words = num_blocks / 32 + (num_blocks % 32 != 0);
    return (words + kSetCtas - 1) / kSetCtas;
}

// OWN: every CTA sets bits in a whole map of its own, and the parts are joined afterwards: atomics on
// another CTA's memory cost far more than those on the CTA's own.  Otherwise (the maps of a pool
// too large for that) a CTA has its part alone, and bits are set where they belong.
template <bool OWN>
__device__ __forceinline__ void set_bit(cg::cluster_group& cluster, uint32_t* map, int32_t words, int32_t id)
{
    const int32_t w = id >> 5;
    const uint32_t bit = 1u << (id & 31);
    if (OWN) {
        atomicOr(map + w, bit);
    } else {
        const int32_t rank = w / words;
        atomicOr(cluster.map_shared_rank(map, rank) + (w - rank * words), bit);
    }
}

// This CTA's part of a map, with the bits that all CTAs have set.
template <bool OWN>
__device__ __forceinline__ uint32_t* set_part(cg::cluster_group& cluster, uint32_t* map, int32_t words)
{
    if (!OWN) return map;
    const int rank = static_cast<int>(cluster.block_rank());
    uint32_t* part = map + rank * words;
    for (int32_t i = threadIdx.x; i < words; i += kSetThreads) {
        uint32_t w[kSetCtas];
#pragma unroll
        for (int c = 0; c < kSetCtas; ++c) w[c] = cluster.map_shared_rank(part, c)[i];
        uint32_t all = 0;
#pragma unroll
        for (int c = 0; c < kSetCtas; ++c) all |= w[c];
        part[i] = all;  // no other CTA reads this part
    }
    __syncthreads();
    return part;
}

// Every row's held entries, one warp a row: begin(r, L, other) gives the entries held, from the row's length and
// its entry of `more`; bit(r, id) takes an id of the pool; end(r, out) is told whether ids outside of it were among them.
template <typename Begin, typename Bit, typename End>
__device__ __forceinline__ void for_rows(cg::cluster_group& cluster, int32_t R, const int32_t* seq_len, const int32_t* more,
                                         const int32_t* block_table, int32_t max_blocks, int32_t num_blocks, Begin begin,
                                         Bit bit, End end)
{
    const int lane = threadIdx.x & 31;
    const int32_t w = threadIdx.x / 32 * kSetCtas + static_cast<int32_t>(cluster.block_rank());
    for (int64_t r0 = w; r0 < R; r0 += 32 * kSetWarps) {
        // the next 32 rows' lengths at once
        const int64_t mine = min(r0 + lane * kSetWarps, static_cast<int64_t>(R - 1));
        const int32_t lengths = seq_len[mine], others = more != nullptr ? more[mine] : 0;
        for (int i = 0; i < 32; ++i) {
            const int64_t row = r0 + i * kSetWarps;
            if (row >= R) break;
            const int32_t r = static_cast<int32_t>(row);
            const int32_t held = begin(r, __shfl_sync(0xFFFFFFFFu, lengths, i), __shfl_sync(0xFFFFFFFFu, others, i));
            const int32_t* table = block_table + row * max_blocks;
            bool out = false;
            for (int32_t e0 = lane; e0 < held; e0 += 32 * kSetBatch) {
                int32_t id[kSetBatch];
#pragma unroll
                for (int q = 0; q < kSetBatch; ++q) id[q] = e0 + 32 * q < held ? table[e0 + 32 * q] : 0;
#pragma unroll
                for (int q = 0; q < kSetBatch; ++q) {
                    if (e0 + 32 * q >= held) continue;
                    if (id[q] >= 0 && id[q] < num_blocks)
                        bit(r, id[q]);
                    else
                        out = true;
                }
            }
            end(r, __any_sync(0xFFFFFFFFu, out));
        }
    }
}

// Exclusive prefix sum of v over the cluster's threads, and its total.  `s_warp` [32], `s_all` [kSetCtas].
__device__ __forceinline__ int32_t cluster_prefix(cg::cluster_group& cluster, int32_t v, int32_t* s_warp, int32_t* s_all,
                                                  int32_t& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int32_t in = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t up = __shfl_up_sync(0xFFFFFFFFu, in, d);
        if (lane >= d) in += up;
    }
    __syncthreads();
    if (lane == 31) s_warp[w] = in;
    __syncthreads();
    int32_t mine = s_warp[lane], run = mine;  // 32 warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t up = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (lane >= d) run += up;
    }
    const int32_t before = __shfl_sync(0xFFFFFFFFu, run - mine, w), cta = __shfl_sync(0xFFFFFFFFu, run, 31);
    const int rank = static_cast<int>(cluster.block_rank());
    if (threadIdx.x < kSetCtas) *(cluster.map_shared_rank(s_all, threadIdx.x) + rank) = cta;
    cluster.sync();
    int32_t ahead = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kSetCtas; ++i) {
        const int32_t x = s_all[i];
        if (i < rank) ahead += x;
        total += x;
    }
    return ahead + before + in - v;
}

// One cluster of kSetCtas CTAs, more than every device lets a kernel have without asking.
template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), const Args& a, int bytes, cudaStream_t stream)
{
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
    if (cudaError_t e = allow_shared(kernel, bytes)) return e;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kSetCtas;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(kSetCtas);
    config.blockDim = dim3(kSetThreads);
    config.dynamicSmemBytes = static_cast<size_t>(bytes);
    config.stream = stream;
    config.attrs = &cluster;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, a);
}

// ---- free -------------------------------------------------------------------
// Bound by latency and by what one cluster can set: 15.5 us for 1,024 rows with 195,000 entries and a stack of
// 150,000 (74 us with a part of the map in each of 8 CTAs and single loads), 6.2 us for 8 rows.
template <bool OWN>
__global__ void __launch_bounds__(kSetThreads) cache_free_kernel(const __grid_constant__ FreeArgs a)
{
    extern __shared__ uint32_t s_set[];
    __shared__ int32_t s_warp[32], s_all[kSetCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const int32_t words = set_words(a.num_blocks), map = OWN ? words * kSetCtas : words;
    uint32_t* s_stay = s_set;        // held by a request that stays, or free already
    uint32_t* s_gone = s_set + map;  // held by one that leaves
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = static_cast<int>(cluster.block_rank());
    for (int32_t i = tid; i < 2 * map; i += kSetThreads) s_set[i] = 0;
    const int32_t count = min(max(a.free_count[0], 0), a.num_blocks);
    if (OWN)
        __syncthreads();
    else
        cluster.sync();

    for (int32_t i0 = rank * kSetThreads + tid; i0 < count; i0 += kSetCtas * kSetThreads * kSetBatch) {
        int32_t id[kSetBatch];
#pragma unroll
        for (int q = 0; q < kSetBatch; ++q) {
            const int64_t i = i0 + static_cast<int64_t>(q) * kSetCtas * kSetThreads;
            id[q] = i < count ? a.free_blocks[i] : -1;
        }
#pragma unroll
        for (int q = 0; q < kSetBatch; ++q)
            if (id[q] >= 0 && id[q] < a.num_blocks) set_bit<OWN>(cluster, s_stay, words, id[q]);
    }
    const int64_t room = static_cast<int64_t>(a.max_blocks) * a.block_size;
    bool leaves = false, bad = false;
    int32_t L = 0;
    for_rows(
        cluster, a.R, a.seq_len, a.leave, a.block_table, a.max_blocks, a.num_blocks,
        [&](int32_t, int32_t length, int32_t leave) {
            L = length;
            leaves = leave != 0;
            bad = L < 0 || L > room;
            const int64_t tokens = bad && (leaves || L < 0) ? 0 : min(static_cast<int64_t>(L), room);
            return tokens > 0 ? a.by_block.quotient(static_cast<int32_t>(tokens - 1)) + 1 : 0;
        },
        [&](int32_t, int32_t id) { set_bit<OWN>(cluster, leaves ? s_gone : s_stay, words, id); },
        [&](int32_t r, bool out) {
            if (lane != 0) return;
            a.seq_len_out[r] = leaves && !bad ? 0 : L;
            if (a.status != nullptr) a.status[r] = (bad ? SV_ST_BAD_LENGTH : 0) | (out ? SV_ST_BAD_BLOCK : 0);
        });
    cluster.sync();

    s_stay = set_part<OWN>(cluster, s_stay, words);
    s_gone = set_part<OWN>(cluster, s_gone, words);
    const int32_t per = (words + kSetThreads - 1) / kSetThreads;
    const int32_t w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int32_t mine = 0, total;
    for (int32_t w = w0; w < w1; ++w) mine += __popc(s_gone[w] & ~s_stay[w]);
    int32_t at = count + cluster_prefix(cluster, mine, s_warp, s_all, total);
    for (int32_t w = w0; w < w1; ++w)
        for (uint32_t bits = s_gone[w] & ~s_stay[w]; bits != 0; bits &= bits - 1) {
            if (at < a.num_blocks) a.free_blocks[at] = (rank * words + w) * 32 + __ffs(bits) - 1;
            ++at;
        }
    if (rank == 0 && tid == 0) a.free_count_out[0] = min(count + total, a.num_blocks);
}

// ---- compact ----------------------------------------------------------------
// The workspace: moves, held blocks U, then the gaps below U in order, the high blocks in
// order, and each high block's number in that order.
struct CompactPlan {
    int32_t* head;
    int32_t *gap, *high, *number;
};
__host__ __device__ inline CompactPlan plan_of(const CompactArgs& a)
{
    int32_t* p = static_cast<int32_t*>(a.workspace);
    const int64_t n = a.cache.num_blocks;
    return CompactPlan{p, p + 64, p + 64 + n, p + 64 + 2 * n};
}

template <bool OWN>
__global__ void __launch_bounds__(kSetThreads) compact_plan_kernel(const __grid_constant__ CompactArgs a)
{
    extern __shared__ uint32_t s_set[];
    __shared__ int32_t s_warp[32], s_all[kSetCtas], s_all2[kSetCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const int32_t N = a.cache.num_blocks, words = set_words(N);
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = static_cast<int>(cluster.block_rank());
    const CompactPlan plan = plan_of(a);
    for (int32_t i = tid; i < (OWN ? words * kSetCtas : words); i += kSetThreads) s_set[i] = 0;
    if (OWN)
        __syncthreads();
    else
        cluster.sync();

    const int64_t room = static_cast<int64_t>(a.max_blocks) * a.cache.block_size;
    bool bad = false;
    for_rows(
        cluster, a.R, a.seq_len, nullptr, a.block_table, a.max_blocks, N,
        [&](int32_t, int32_t L, int32_t) {
            const int32_t tokens = static_cast<int32_t>(min(static_cast<int64_t>(max(L, 0)), room));
            bad = L != tokens;
            return tokens > 0 ? a.by_block.quotient(tokens - 1) + 1 : 0;
        },
        [&](int32_t, int32_t id) { set_bit<OWN>(cluster, s_set, words, id); },
        [&](int32_t r, bool out) {
            if (lane == 0 && a.status != nullptr) a.status[r] = (bad ? SV_ST_BAD_LENGTH : 0) | (out ? SV_ST_BAD_BLOCK : 0);
        });
    cluster.sync();

    const uint32_t* part = set_part<OWN>(cluster, s_set, words);
    const int32_t per = (words + kSetThreads - 1) / kSetThreads;
    const int32_t w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int32_t mine = 0, U;
    for (int32_t w = w0; w < w1; ++w) mine += __popc(part[w]);
    const int32_t before = cluster_prefix(cluster, mine, s_warp, s_all, U);  // held blocks before word w0
    // Of the ids below U as many are gaps as there are held ones at U or above.  A held id x >= U with h held
    // ids below it is move h - (held ids below U); a gap x < U with h held ids below it is move x - h.
    int32_t low = 0, below;
    for (int32_t w = w0; w < w1; ++w) {
        const int32_t id = (rank * words + w) * 32, left = U - id;
        low += __popc(left >= 32 ? part[w] : left <= 0 ? 0u : part[w] & ((1u << left) - 1));
    }
    cluster_prefix(cluster, low, s_warp, s_all2, below);
    int32_t h = before;
    for (int32_t w = w0; w < w1; ++w) {
        const uint32_t bits = part[w];
        const int32_t id = (rank * words + w) * 32;
        for (int32_t i = 0; i < 32 && id + i < N; ++i) {
            const bool held = (bits >> i) & 1u;
            const int32_t x = id + i;
            if (held && x >= U) {
                plan.high[h - below] = x;
                plan.number[x] = h - below;
            }
            if (!held && x < U) plan.gap[x - h] = x;
            h += held;
        }
    }
    if (rank == 0 && tid == 0) {
        plan.head[0] = U - below;
        plan.head[1] = U;
        a.free_count[0] = N - U;
    }
}

constexpr int kPackThreads = 256;

// How the 16-byte vectors of a block's plane (one layer's K or V) lie, in rising order of stride.
struct PackGeom {
    int32_t vecs, inner, outer;          // vectors of a head, then the axis with the smaller stride, then the other
    Divisor by_vecs, by_inner;
    int64_t inner_stride, outer_stride;  // elements
    int32_t total, pieces;               // vectors of a plane, thread blocks' pieces of it
    uint32_t planes;
};

// Bound by bytes: 238 us for both kernels where 751 MB move (1,502 MB read and written), 6.3 TB/s, 0.93 of a copy's rate,
// of which the plan takes 10 (the moves alone run at the copy's rate); 11 us for a small pool.
__global__ void __launch_bounds__(kPackThreads) compact_move_kernel(const CompactArgs a, const PackGeom g)
{
    const CompactPlan plan = plan_of(a);
    const int tid = threadIdx.x;
    const int32_t moves = plan.head[0], U = plan.head[1], N = a.cache.num_blocks;
    const int64_t threads = static_cast<int64_t>(gridDim.x) * kPackThreads, me = static_cast<int64_t>(blockIdx.x) * kPackThreads + tid;

    // tables and the stack
    const int64_t entries = static_cast<int64_t>(a.R) * a.max_blocks;
    for (int64_t i = me; i < entries; i += threads) {
        const int32_t r = static_cast<int32_t>(i / a.max_blocks), c = static_cast<int32_t>(i - static_cast<int64_t>(r) * a.max_blocks);
        const int64_t L = a.seq_len[r];
        int32_t id = -1;
        if (static_cast<int64_t>(c) * a.cache.block_size < L) {
            id = a.block_table[i];
            if (id >= U && id < N) id = plan.gap[plan.number[id]];
        }
        a.block_table_out[i] = id;
    }
    for (int64_t i = me; i < N; i += threads) a.free_blocks[i] = i < N - U ? static_cast<int32_t>(N - 1 - i) : -1;

    // pieces of moves
    const int64_t units = static_cast<int64_t>(moves) * g.planes * g.pieces;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int32_t piece = static_cast<int32_t>(unit % g.pieces);
        const int64_t rest = unit / g.pieces;
        const uint32_t plane = static_cast<uint32_t>(rest % g.planes);
        const int32_t move = static_cast<int32_t>(rest / g.planes);
        uint16_t* p = static_cast<uint16_t*>((plane & 1) ? a.cache.v : a.cache.k) + static_cast<int64_t>(plane >> 1) * a.cache.layer_stride;
        const uint16_t* src = p + plan.high[move] * a.cache.block_stride;
        uint16_t* dst = p + plan.gap[move] * a.cache.block_stride;
        const int32_t v0 = piece * (kPackThreads * kMoveBatch) + tid;
        uint4 val[kMoveBatch];
        int64_t at[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int32_t v = v0 + u * kPackThreads;
            const int32_t head = g.by_vecs.quotient(v), outer = g.by_inner.quotient(head);
            at[u] = (head - outer * g.inner) * g.inner_stride + outer * g.outer_stride + (v - head * g.vecs) * 8;
            if (v < g.total) val[u] = *reinterpret_cast<const uint4*>(src + at[u]);
        }
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (v0 + u * kPackThreads < g.total) *reinterpret_cast<uint4*>(dst + at[u]) = val[u];
    }
}

}  // namespace

cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t stream)
{
    const int64_t columns = 2ll * a.cache.layers * a.cache.kv_heads * (a.cache.head_dim / 8);
    const int64_t rows = (columns + kForkThreads - 1) / kForkThreads;
    // few rows leave room for several thread blocks to a last block's tokens; those of rows that fork nothing cost, too
    const int64_t shares = std::min<int64_t>((a.cache.block_size + kMoveBatch - 1) / kMoveBatch,
                                             std::max<int64_t>(1, 64ll * std::max(1, device_sm_count()) / (a.R * rows)));
    const dim3 grid(static_cast<unsigned>(a.R), static_cast<unsigned>(rows), static_cast<unsigned>(std::min<int64_t>(shares, 65535)));
    cache_fork_kernel<<<grid, kForkThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_free(const FreeArgs& a, cudaStream_t stream)
{
    const int part = 2 * 4 * set_words(a.num_blocks), whole = part * kSetCtas;
    return whole <= kSetOwnBytes ? launch_cluster(cache_free_kernel<true>, a, whole, stream)
                                 : launch_cluster(cache_free_kernel<false>, a, part, stream);
}

size_t compact_workspace_bytes(int32_t num_blocks) { return 256 + 12 * static_cast<size_t>(num_blocks); }

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream)
{
    const int part = 4 * set_words(a.cache.num_blocks), whole = part * kSetCtas;
    if (cudaError_t e = whole <= kSetOwnBytes ? launch_cluster(compact_plan_kernel<true>, a, whole, stream)
                                              : launch_cluster(compact_plan_kernel<false>, a, part, stream))
        return e;
    PackGeom g{};
    g.vecs = a.cache.head_dim / 8;
    const bool heads_in = a.cache.kv_heads == 1 || a.cache.head_stride <= a.cache.token_stride;
    g.inner = heads_in ? a.cache.kv_heads : a.cache.block_size;
    g.outer = heads_in ? a.cache.block_size : a.cache.kv_heads;
    g.inner_stride = heads_in ? a.cache.head_stride : a.cache.token_stride;
    g.outer_stride = heads_in ? a.cache.token_stride : a.cache.head_stride;
    g.by_vecs = divisor_of(g.vecs);
    g.by_inner = divisor_of(g.inner);
    g.total = g.vecs * g.inner * g.outer;
    g.pieces = (g.total + kPackThreads * kMoveBatch - 1) / (kPackThreads * kMoveBatch);
    g.planes = 2u * a.cache.layers;
    compact_move_kernel<<<8 * std::max(1, device_sm_count()), kPackThreads, 0, stream>>>(a, g);
    return cudaGetLastError();
}

}  // namespace sv
