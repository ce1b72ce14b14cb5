// The bookkeeping around a verify step over a paged cache: step_tables_kernel
// lays the step's tokens out (blocks, slots, positions, ancestor masks) and
// cache_commit_kernel keeps the accepted path and gives surplus blocks back.
//
// Both answer prefix sums over the requests without a second launch or a grid
// barrier: a CTA needs only the sums before its own range of requests, which it
// takes by one block reduction over the lengths (4 to 8 bytes a request, from L2).
#include <algorithm>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepWarps = kStepThreads / 32;

__device__ __forceinline__ int64_t warp_sum(int64_t v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Sums of a and b over the block; every thread gets them.  `s` holds 2 * kStepWarps values.
__device__ __forceinline__ void block_sum2(int64_t& a, int64_t& b, int64_t* s)
{
    a = warp_sum(a);
    b = warp_sum(b);
    const int w = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        s[2 * w] = a;
        s[2 * w + 1] = b;
    }
    __syncthreads();
    a = 0;
    b = 0;
#pragma unroll
    for (int i = 0; i < kStepWarps; ++i) {
        a += s[2 * i];
        b += s[2 * i + 1];
    }
}

// Exclusive prefix sums of a and b over the block's threads; `s` as above.
__device__ __forceinline__ void block_prefix2(int64_t& a, int64_t& b, int64_t* s)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t ua = __shfl_up_sync(0xFFFFFFFFu, ia, d), ub = __shfl_up_sync(0xFFFFFFFFu, ib, d);
        if (lane >= d) {
            ia += ua;
            ib += ub;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s[2 * w] = ia;
        s[2 * w + 1] = ib;
    }
    __syncthreads();
    a = ia - a;
    b = ib - b;
    for (int i = 0; i < w; ++i) {
        a += s[2 * i];
        b += s[2 * i + 1];
    }
}

// blocks that hold `tokens` tokens, 0 <= tokens < 2^31
__device__ __forceinline__ int32_t blocks_of(int32_t tokens, const Divisor& by_block)
{
    return tokens > 0 ? by_block.quotient(tokens - 1) + 1 : 0;
}

// What one request asks for.
struct Ask {
    int32_t tokens;  // new tokens, 0 for a negative length
    int32_t held, need;
    bool bad;  // a length that the tables cannot hold
};

__device__ __forceinline__ Ask ask_of(const StepTablesArgs& a, int32_t r)
{
    const int32_t L = a.seq_len[r], n = a.new_len[r];
    Ask q;
    q.tokens = max(n, 0);
    const int64_t total = static_cast<int64_t>(L) + n;
    q.bad = L < 0 || n < 0 || total > static_cast<int64_t>(a.max_blocks) * a.block_size ||
            (a.parent != nullptr && (n > SV_MAX_TREE || n > 32 * static_cast<int64_t>(a.mask_words)));
    q.held = q.bad ? 0 : blocks_of(L, a.by_block);
    q.need = q.bad ? 0 : blocks_of(static_cast<int32_t>(total), a.by_block) - q.held;
    return q;
}

// A thread takes one token at a time.  The ancestors of a token are visited in
// falling order of their number (a parent lies below its child), so the words of
// its mask come out one after the other, from the highest to the lowest, without
// any storage beyond the word in hand.
// Bound by latency: the sums over the lengths before a CTA's range with their block reductions, a
// block's ids, then the words of the masks.  11.9 us for 1,024 requests of 65 tokens (1.9 MB), 3 for
// one of 9; the parts have not been timed apart.
__global__ void __launch_bounds__(kStepThreads) step_tables_kernel(const StepTablesArgs a)
{
    __shared__ int64_t s_sum[2 * kStepWarps];
    __shared__ int32_t s_parent[SV_MAX_TREE];
    const int tid = threadIdx.x;
    const int64_t grid = gridDim.x;
    const int32_t r0 = static_cast<int32_t>(static_cast<int64_t>(a.R) * blockIdx.x / grid);
    const int32_t r1 = static_cast<int32_t>(static_cast<int64_t>(a.R) * (blockIdx.x + 1) / grid);
    const int64_t count = min(max(a.free_count[0], 0), a.num_blocks);

    int64_t cum = 0, pre = 0;  // tokens and blocks asked for before request r0
    for (int32_t r = tid; r < r0; r += kStepThreads) {
        const Ask q = ask_of(a, r);
        cum += q.tokens;
        pre += q.need;
    }
    block_sum2(cum, pre, s_sum);
    if (blockIdx.x == 0 && tid == 0) a.cu_tokens[0] = 0;

    for (int32_t r = r0; r < r1; ++r) {
        const Ask q = ask_of(a, r);
        const int32_t L = a.seq_len[r];
        const int64_t end = cum + q.tokens;
        const bool full = !q.bad && ((q.need > 0 && pre + q.need > count) || (q.tokens > 0 && end > a.T));
        const bool takes = !q.bad && !full;
        const int32_t t0 = static_cast<int32_t>(min(cum, static_cast<int64_t>(a.T)));
        const int32_t t1 = static_cast<int32_t>(min(end, static_cast<int64_t>(a.T)));
        int32_t* table = a.block_table + static_cast<int64_t>(r) * a.max_blocks;
        uint32_t st = q.bad ? SV_ST_BAD_LENGTH : full ? SV_ST_NO_BLOCKS : 0u;
        const bool tree = a.parent != nullptr && takes;
        if (tree) {
            __syncthreads();  // the request before this one has read its parents
            for (int32_t j = tid; j < t1 - t0; j += kStepThreads) s_parent[j] = a.parent[t0 + j];
            __syncthreads();
        }
        if (takes)
            for (int32_t i = tid; i < q.need; i += kStepThreads)
                table[q.held + i] = a.free_blocks[count - 1 - (pre + i)];
        for (int32_t j = tid; j < t1 - t0; j += kStepThreads) {
            int64_t slot = -1;
            if (takes) {
                const int32_t at = L + j, b = a.by_block.quotient(at);
                const int32_t id = b < q.held ? table[b] : a.free_blocks[count - 1 - (pre + b - q.held)];
                if (id >= 0 && id < a.num_blocks)
                    slot = static_cast<int64_t>(id) * a.block_size + (at - b * a.block_size);
                else
                    st |= SV_ST_BAD_BLOCK;
            }
            a.slot[t0 + j] = slot;
            int32_t depth = j;
            if (tree) {
                uint32_t* row = a.mask + static_cast<int64_t>(t0 + j) * a.mask_words;
                int32_t w = a.mask_words - 1;
                uint32_t word = 0;
                depth = -1;
                for (int32_t x = j; x >= 0;) {
                    for (; w > (x >> 5); --w) {
                        row[w] = word;
                        word = 0;
                    }
                    word |= 1u << (x & 31);
                    ++depth;
                    const int32_t p = s_parent[x];
                    if (p >= x || p < -1) {
                        st |= SV_ST_BAD_TREE;
                        break;
                    }
                    x = p;
                }
                for (; w >= 0; --w) {
                    row[w] = word;
                    word = 0;
                }
            } else if (a.parent != nullptr) {
                for (int32_t w = 0; w < a.mask_words; ++w)
                    a.mask[static_cast<int64_t>(t0 + j) * a.mask_words + w] = 0;
            }
            a.position[t0 + j] = takes ? L + depth : -1;
        }
        st = __syncthreads_or(static_cast<int>(st & SV_ST_BAD_TREE)) ? st | SV_ST_BAD_TREE : st;
        st = __syncthreads_or(static_cast<int>(st & SV_ST_BAD_BLOCK)) ? st | SV_ST_BAD_BLOCK : st;
        if (tid == 0) {
            a.cu_tokens[r + 1] = t1;
            a.kv_len[r] = takes ? L + q.tokens : 0;
            if (a.status != nullptr) a.status[r] = static_cast<int32_t>(st);
        }
        cum = end;
        pre += q.need;
    }
    if (blockIdx.x + 1 != gridDim.x) return;

    // The last CTA: entries behind the last token, and the blocks that are left.  From the first
    // request that does not fit no request takes blocks, so what is taken is the blocks asked for
    // before that one (all of them where every request fits).
    for (int64_t t = min(cum, static_cast<int64_t>(a.T)) + tid; t < a.T; t += kStepThreads) {
        a.slot[t] = -1;
        a.position[t] = -1;
        if (a.parent != nullptr)
            for (int32_t w = 0; w < a.mask_words; ++w) a.mask[t * a.mask_words + w] = 0;
    }
    int64_t taken = pre;
    if (pre > count || cum > a.T) {
        const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(a.R) * tid / kStepThreads);
        const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(a.R) * (tid + 1) / kStepThreads);
        int64_t tok = 0, blk = 0;
        for (int32_t r = c0; r < c1; ++r) {
            const Ask q = ask_of(a, r);
            tok += q.tokens;
            blk += q.need;
        }
        block_prefix2(tok, blk, s_sum);
        int64_t mine = 0;
        for (int32_t r = c0; r < c1; ++r) {
            const Ask q = ask_of(a, r);
            tok += q.tokens;
            blk += q.need;
            if (!q.bad && blk <= count && tok <= a.T) mine += q.need;
        }
        int64_t none = 0;
        block_sum2(mine, none, s_sum);
        taken = mine;
    }
    if (tid == 0) a.free_count_out[0] = static_cast<int32_t>(count - taken);
}

// ---- commit -----------------------------------------------------------------
// What a request keeps.
struct Keep {
    int32_t root, n, a;  // seq_len, tokens of this step, accepted drafts
    bool takes, bad;
    int32_t held, kept;  // blocks before and after
};

__device__ __forceinline__ int32_t path_at(const CommitArgs& c, int32_t r, int32_t i)
{
    if (c.path != nullptr) return c.path[static_cast<int64_t>(r) * c.k + i];
    const int64_t b = c.branch != nullptr ? c.branch[r] : 0;
    const int64_t x = 1 + b * c.k + i;
    return x < 1 || x > INT32_MAX ? -1 : static_cast<int32_t>(x);
}

__device__ __forceinline__ Keep keep_of(const CommitArgs& c, int32_t r)
{
    Keep q;
    q.root = c.seq_len[r];
    q.n = c.cu_tokens[r + 1] - c.cu_tokens[r];
    const int32_t kv = c.kv_len[r], accepted = c.accept_len[r];  // loaded with the lengths before
    const int64_t room = static_cast<int64_t>(c.max_blocks) * c.cache.block_size;
    q.takes = q.root >= 0 && q.n > 0 && static_cast<int64_t>(q.root) + q.n == kv && kv <= room;
    q.a = q.takes ? min(max(accepted, 0), c.k) : 0;
    q.bad = false;
    if (c.path != nullptr) {
        int32_t last = 0;
        for (int32_t i = 0; i < q.a; ++i) {
            const int32_t x = path_at(c, r, i);
            if (x <= last || x >= q.n) {
                q.a = i;
                q.bad = true;
            } else {
                last = x;
            }
        }
    } else if (q.a > 0) {  // consecutive tokens: only the ends can lie outside
        const int32_t x = path_at(c, r, 0);
        const int32_t most = x < 1 ? 0 : max(0, min(q.a, q.n - x));
        q.bad = most < q.a;
        q.a = most;
    }
    q.held = q.takes ? blocks_of(kv, c.by_block) : 0;
    q.kept = q.takes ? blocks_of(q.root + 1 + q.a, c.by_block) : 0;
    return q;
}

// What a request gives back: the blocks behind the ones it keeps, of which only ids of the pool go on the
// free list, as any request may get them from there.  `bad`: a block of the step's tokens is outside the pool.
struct Surplus {
    int32_t blocks;
    bool bad;
};

__device__ __forceinline__ bool in_pool(const CommitArgs& c, int32_t id) { return id >= 0 && id < c.cache.num_blocks; }

__device__ __forceinline__ Surplus surplus_of(const CommitArgs& c, int32_t r, const Keep& q)
{
    Surplus s{0, false};
    const int32_t* table = c.block_table + static_cast<int64_t>(r) * c.max_blocks;
    for (int32_t b = q.takes ? c.by_block.quotient(q.root) : q.held; b < q.held; ++b) {
        const bool in = in_pool(c, table[b]);
        s.bad = s.bad || !in;
        s.blocks += in && b >= q.kept;
    }
    return s;
}

constexpr int kMoveBatch = 8;

// Grid: x = requests, then the CTAs that give blocks back; y = 128 16-byte columns of
// the heads of all layers, K and V.  A thread owns a column and walks the path upward,
// eight tokens' loads before their stores.  That order is safe in place: the i-th
// destination is token 1 + i, the path increases, so a token still to be read
// (number >= 1 + its index) is never below the ones already written.  The places are
// looked up once per CTA, all at a time, so that a round is one trip to memory.
// Bound by the latency of a path's ceil(a / 8) rounds for few requests and by memory
// for many: 9.9 us for 64 requests over 16 layers, 34 MB, 3.4 TB/s (20 us with the places
// looked up token by token), 8.0 where they lie in L2; 3.3 us for 4 requests over 4 layers.  By path
// every thread checks the whole path: 16.6 us from a cold L2, where a branch takes 11.5.
__global__ void __launch_bounds__(kStepThreads) cache_commit_kernel(const CommitArgs c, int32_t releasers)
{
    __shared__ int64_t s_sum[2 * kStepWarps];
    const int tid = threadIdx.x;
    if (static_cast<int32_t>(blockIdx.x) >= c.R) {
        if (blockIdx.y != 0) return;
        const int32_t i = static_cast<int32_t>(blockIdx.x) - c.R;
        const int32_t r0 = static_cast<int32_t>(static_cast<int64_t>(c.R) * i / releasers);
        const int32_t r1 = static_cast<int32_t>(static_cast<int64_t>(c.R) * (i + 1) / releasers);
        const int64_t count = min(max(c.free_count[0], 0), c.cache.num_blocks);
        int64_t before = 0, none = 0;
        for (int32_t r = tid; r < r0; r += kStepThreads) before += surplus_of(c, r, keep_of(c, r)).blocks;
        block_sum2(before, none, s_sum);
        int64_t top = count + before;
        for (int32_t base = r0; base < r1; base += kStepThreads) {
            const int32_t r = base + tid;
            Keep q{};
            Surplus give{};
            if (r < r1) {
                q = keep_of(c, r);
                give = surplus_of(c, r, q);
            }
            int64_t mine = give.blocks, all = mine, zero = 0;
            block_prefix2(mine, zero, s_sum);
            __syncthreads();
            int64_t at = top + mine;
            if (r < r1) {
                const int32_t* table = c.block_table + static_cast<int64_t>(r) * c.max_blocks;
                for (int32_t b = q.kept; b < q.held; ++b) {
                    const int32_t id = table[b];
                    if (!in_pool(c, id)) continue;
                    if (at < c.cache.num_blocks) c.free_blocks[at] = id;
                    ++at;
                }
                c.seq_len_out[r] = q.takes ? q.root + 1 + q.a : q.root;
                if (c.status != nullptr) c.status[r] = (q.bad ? SV_ST_BAD_TREE : 0) | (give.bad ? SV_ST_BAD_BLOCK : 0);
            }
            zero = 0;
            block_sum2(all, zero, s_sum);
            top += all;
        }
        if (i + 1 == releasers && tid == 0)
            c.free_count_out[0] = static_cast<int32_t>(min(top, static_cast<int64_t>(c.cache.num_blocks)));
        return;
    }

    const int32_t r = blockIdx.x;
    if (c.path == nullptr && (c.branch == nullptr || c.branch[r] == 0)) return;  // they lie where they belong
    const Keep q = keep_of(c, r);
    if (q.a == 0) return;
    __shared__ int64_t s_src[SV_MAX_K], s_dst[SV_MAX_K];
    const int32_t* table = c.block_table + static_cast<int64_t>(r) * c.max_blocks;
    auto place = [&](int32_t token) -> int64_t {
        const int32_t at = q.root + token, b = c.by_block.quotient(at), id = table[b];
        if (!in_pool(c, id)) return -1;
        return id * c.cache.block_stride + (at - b * c.cache.block_size) * c.cache.token_stride;
    };
    for (int32_t i = tid; i < q.a; i += kStepThreads) {
        const int32_t x = path_at(c, r, i);
        const int64_t src = place(x), dst = place(1 + i);
        s_src[i] = src;
        s_dst[i] = src < 0 || x == 1 + i ? -1 : dst;
    }
    __syncthreads();
    const int32_t vecs = c.cache.head_dim / 8, columns = c.cache.kv_heads * vecs;
    const int64_t column = static_cast<int64_t>(blockIdx.y) * kStepThreads + tid;
    const int32_t plane = static_cast<int32_t>(column / columns), col = static_cast<int32_t>(column - static_cast<int64_t>(plane) * columns);
    if (plane >= 2 * c.cache.layers) return;
    const int32_t h = col / vecs;
    uint16_t* p = static_cast<uint16_t*>((plane & 1) ? c.cache.v : c.cache.k) + (plane >> 1) * c.cache.layer_stride +
                  h * c.cache.head_stride + (col - h * vecs) * 8;
    for (int32_t i0 = 0; i0 < q.a; i0 += kMoveBatch) {
        uint4 val[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (i0 + u < q.a && s_dst[i0 + u] >= 0) val[u] = *reinterpret_cast<const uint4*>(p + s_src[i0 + u]);
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (i0 + u < q.a && s_dst[i0 + u] >= 0) *reinterpret_cast<uint4*>(p + s_dst[i0 + u]) = val[u];
    }
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream)
{
    const int32_t most = std::max(1, device_sm_count()) * 8;
    step_tables_kernel<<<std::min(a.R, most), kStepThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_commit(const CommitArgs& a, cudaStream_t stream)
{
    const int32_t releasers = std::min(32, (a.R + kStepThreads - 1) / kStepThreads);
    const int64_t columns = 2ll * a.cache.layers * a.cache.kv_heads * (a.cache.head_dim / 8);
    const int64_t rows = (columns + kStepThreads - 1) / kStepThreads;
    if (rows > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(a.R) + releasers, static_cast<unsigned>(rows));
    cache_commit_kernel<<<grid, kStepThreads, 0, stream>>>(a, releasers);
    return cudaGetLastError();
}

}  // namespace sv
