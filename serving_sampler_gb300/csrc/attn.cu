// sv_tree_attention: softmax(scale q k^T) v of the step's tokens over the paged
// cache, a first form: one CTA takes one token's query head and walks its keys
// 128 at a time with a running maximum and sum (one pass over K and V).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kAttnThreads = 128;

template <bool F16>
__device__ __forceinline__ float entry_f(uint16_t w)
{
    return F16 ? __half2float(__ushort_as_half(w)) : __uint_as_float(static_cast<uint32_t>(w) << 16);
}

template <bool F16>
__global__ void __launch_bounds__(kAttnThreads) tree_attention_kernel(const AttnArgs a)
{
    __shared__ float s_q[SV_MAX_HEAD_DIM];
    __shared__ float s_p[kAttnThreads];
    __shared__ int64_t s_at[kAttnThreads];
    __shared__ float s_red[kAttnThreads / 32];
    const int tid = threadIdx.x;
    const int32_t t = blockIdx.x, h = blockIdx.y;
    const int32_t T = a.q.tokens, D = a.q.head_dim;
    // the request of this token
    int32_t lo = 0, hi = a.R;
    while (lo < hi) {
        const int32_t mid = (lo + hi) / 2;
        if (min(max(a.cu_tokens[mid + 1], 0), T) <= t) lo = mid + 1;
        else hi = mid;
    }
    if (lo == a.R) return;
    const int32_t r = lo;
    const int32_t t0 = min(max(a.cu_tokens[r], 0), T), n = min(max(a.cu_tokens[r + 1], 0), T) - t0, i = t - t0;
    if (i < 0 || i >= a.max_tokens) return;
    const int32_t kv = min(max(a.kv_len[r], 0), a.max_blocks * a.cache.block_size), ctx = kv - n;
    const int32_t hk = h / (a.q.heads / a.cache.kv_heads);
    const uint16_t* q = static_cast<const uint16_t*>(a.q.data) + t * a.q.token_stride + h * a.q.head_stride;
    const uint16_t* K = static_cast<const uint16_t*>(a.cache.k) + hk * a.cache.head_stride;
    const uint16_t* V = static_cast<const uint16_t*>(a.cache.v) + hk * a.cache.head_stride;
    if (tid < D) s_q[tid] = entry_f<F16>(q[tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int32_t x0 = 0; x0 < kv; x0 += kAttnThreads) {
        const int32_t x = x0 + tid;
        bool see = x < kv;
        if (see && x >= ctx) {
            const int32_t j = x - ctx;
            if (a.mask == nullptr) see = j <= i;
            else see = j < 32 * a.mask_words && ((a.mask[static_cast<int64_t>(t) * a.mask_words + j / 32] >> (j % 32)) & 1);
        }
        float s = -INFINITY;
        int64_t at = -1;
        if (see) {
            const int32_t b = x / a.cache.block_size;
            const int32_t id = a.block_table[static_cast<int64_t>(r) * a.max_blocks + b];
            s = 0.0f;
            if (id >= 0 && id < a.cache.num_blocks) {
                at = static_cast<int64_t>(id) * a.cache.block_stride + static_cast<int64_t>(x - b * a.cache.block_size) * a.cache.token_stride;
                for (int32_t d = 0; d < D; ++d) s = fmaf(s_q[d], entry_f<F16>(K[at + d]), s);
            }
            s *= a.scale;
        }
        float top = s;
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if ((tid & 31) == 0) s_red[tid >> 5] = top;
        __syncthreads();
        for (int w = 0; w < kAttnThreads / 32; ++w) top = fmaxf(top, s_red[w]);
        const float m2 = fmaxf(m, top), ref = m2 == -INFINITY ? 0.0f : m2;
        const float back = expf(m - ref);
        const float p = see ? expf(s - ref) : 0.0f;
        s_p[tid] = p;
        s_at[tid] = at;
        float sum = p;
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        __syncthreads();
        if ((tid & 31) == 0) s_red[tid >> 5] = sum;
        __syncthreads();
        sum = s_red[0] + s_red[1] + s_red[2] + s_red[3];
        l = l * back + sum;
        acc *= back;
        if (tid < D)
            for (int c = 0; c < kAttnThreads; ++c)
                if (s_at[c] >= 0) acc = fmaf(s_p[c], entry_f<F16>(V[s_at[c] + tid]), acc);
        m = m2;
        __syncthreads();
    }
    if (tid < D) {
        const float o = l == 0.0f ? 0.0f : acc / l;
        uint16_t* dst = static_cast<uint16_t*>(const_cast<void*>(a.out.data)) + t * a.out.token_stride + h * a.out.head_stride;
        dst[tid] = F16 ? __half_as_ushort(__float2half_rn(o)) : __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
    if (tid == 0 && a.lse != nullptr)
        a.lse[static_cast<int64_t>(t) * a.q.heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
    if (tid == 0 && h == 0 && i == 0 && a.status != nullptr) a.status[r] = 0;
}

}  // namespace

size_t attn_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int64_t) { return 256; }

cudaError_t launch_tree_attention(const AttnArgs& a, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(a.q.tokens), static_cast<unsigned>(a.q.heads));
    if (a.cache.dtype == SV_F16)
        tree_attention_kernel<true><<<grid, kAttnThreads, 0, stream>>>(a);
    else
        tree_attention_kernel<false><<<grid, kAttnThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace sv
