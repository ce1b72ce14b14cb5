// The C ABI of specverify: argument checks, then the kernel launchers.
// Declarations and the contract of every call are in include/specverify.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "specverify.h"
#include "sv_internal.h"

namespace sv {

// A device's SM count does not change: asked for once per device.
int device_sm_count()
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < kDevices && (n = known[dev].load(std::memory_order_relaxed)) != 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Validate a logit matrix with `rows` rows; `min_stride` is the smallest
// legal row stride (the width, or offset + width for CFG partitions).
static int check_rows(const sv_rows& m, int64_t rows, int64_t min_stride, Rows* out)
{
    if (m.dtype != SV_BF16 && m.dtype != SV_F32) return SV_ERR_DTYPE;
    if (m.width < 1 || m.width > SV_MAX_WIDTH) return SV_ERR_SHAPE;
    if (rows > 1 && m.row_stride < min_stride) return SV_ERR_SHAPE;
    if (m.row_stride < 0) return SV_ERR_SHAPE;
    if (rows > 0 && m.data == nullptr) return SV_ERR_INVALID_ARG;
    const int es = m.dtype == SV_BF16 ? 2 : 4;
    if (!aligned(m.data, es)) return SV_ERR_ALIGN;
    out->data = static_cast<const char*>(m.data);
    out->dtype = m.dtype;
    out->esize = es;
    out->width = m.width;
    out->stride = rows > 1 ? m.row_stride : std::max<int64_t>(m.row_stride, min_stride);
    out->bulk_ok = aligned(m.data, 16) && ((out->stride * es) % 16 == 0);
    return SV_OK;
}

static int check_workspace(const void* ws, size_t bytes, size_t need)
{
    if (ws == nullptr || bytes < need || !aligned(ws, 256)) return SV_ERR_WORKSPACE;
    return SV_OK;
}

static int launched(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_LAUNCH; }

static int check_cache(const sv_kv_cache& c, bool data)
{
    if (c.dtype != SV_BF16 && c.dtype != SV_F16) return SV_ERR_DTYPE;
    if (c.num_blocks < 1 || c.block_size < 1 || c.kv_heads < 1 || c.layers < 1 || c.head_dim < 1)
        return SV_ERR_SHAPE;
    if (c.head_dim > SV_MAX_HEAD_DIM) return SV_ERR_LIMIT;
    if (c.head_dim % 8 != 0 || c.block_size % 8 != 0) return SV_ERR_SHAPE;
    // every axis steps by at least one head's entries where it has more than one step
    const int64_t least = c.head_dim;
    if ((c.num_blocks > 1 && c.block_stride < least) || c.token_stride < least ||
        (c.kv_heads > 1 && c.head_stride < least) || (c.layers > 1 && c.layer_stride < least) ||
        c.block_stride < 0 || c.head_stride < 0 || c.layer_stride < 0)
        return SV_ERR_SHAPE;
    if (data && (c.k == nullptr || c.v == nullptr)) return SV_ERR_INVALID_ARG;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || c.token_stride % 8 != 0 ||
        (c.num_blocks > 1 && c.block_stride % 8 != 0) || (c.kv_heads > 1 && c.head_stride % 8 != 0) ||
        (c.layers > 1 && c.layer_stride % 8 != 0))
        return SV_ERR_ALIGN;
    return SV_OK;
}

// Heads of packed tokens that go with `dtype`, `head_dim` and `tokens`.
static int check_heads(const sv_heads& h, int32_t dtype, int32_t head_dim, int32_t tokens)
{
    if (h.dtype != dtype) return SV_ERR_DTYPE;
    if (h.heads < 1 || h.head_dim != head_dim || h.tokens != tokens) return SV_ERR_SHAPE;
    if ((h.tokens > 1 && h.token_stride < head_dim) || (h.heads > 1 && h.head_stride < head_dim) ||
        h.token_stride < 0 || h.head_stride < 0)
        return SV_ERR_SHAPE;
    if (tokens > 0 && h.data == nullptr) return SV_ERR_INVALID_ARG;
    if (!aligned(h.data, 16) || (h.tokens > 1 && h.token_stride % 8 != 0) ||
        (h.heads > 1 && h.head_stride % 8 != 0))
        return SV_ERR_ALIGN;
    return SV_OK;
}

static bool have_device()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess;
}

static int tree_attention(const AttnArgs& a, size_t workspace_bytes, sv_stream_t stream)
{
    if (a.R < 0 || a.q.tokens < 0 || a.max_tokens < 0 || a.max_blocks < 0) return SV_ERR_INVALID_ARG;
    if (a.mask_words < 0 || (a.mask != nullptr && a.mask_words < 1)) return SV_ERR_INVALID_ARG;
    if (int rc = check_cache(a.cache, a.R > 0 && a.q.tokens > 0)) return rc;
    if (a.cache.layers != 1) return SV_ERR_SHAPE;
    if (static_cast<int64_t>(a.max_blocks) * a.cache.block_size > INT32_MAX) return SV_ERR_LIMIT;
    if (a.R == 0 || (a.q.tokens == 0 && a.status == nullptr)) return SV_OK;
    if (a.q.tokens == 0) {  // nothing to attend for, and nothing went wrong
        if (!aligned(a.status, 4)) return SV_ERR_ALIGN;
        if (!have_device()) return SV_ERR_DEVICE;
        return launched(cudaMemsetAsync(a.status, 0, static_cast<size_t>(a.R) * 4, stream));
    }
    if (int rc = check_heads(a.q, a.cache.dtype, a.cache.head_dim, a.q.tokens)) return rc;
    if (int rc = check_heads(a.out, a.cache.dtype, a.cache.head_dim, a.q.tokens)) return rc;
    if (a.out.heads != a.q.heads || a.q.heads % a.cache.kv_heads != 0) return SV_ERR_SHAPE;
    if (a.q.heads / a.cache.kv_heads > SV_MAX_GROUP) return SV_ERR_LIMIT;
    if (a.kv_len == nullptr || a.cu_tokens == nullptr || (a.max_blocks > 0 && a.block_table == nullptr))
        return SV_ERR_INVALID_ARG;
    if (!aligned(a.block_table, 4) || !aligned(a.kv_len, 4) || !aligned(a.cu_tokens, 4) || !aligned(a.mask, 4) ||
        !aligned(a.lse, 4) || !aligned(a.status, 4))
        return SV_ERR_ALIGN;
    if (int rc = check_workspace(a.workspace, workspace_bytes,
                                 attn_workspace_bytes(a.R, a.max_tokens, a.q.heads, a.cache.kv_heads, a.q.head_dim,
                                                      static_cast<int64_t>(a.max_blocks) * a.cache.block_size)))
        return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_tree_attention(a, stream));
}

}  // namespace sv

using namespace sv;

extern "C" {

const char* sv_status_string(int code)
{
    switch (code) {
        case SV_OK: return "ok";
        case SV_ERR_INVALID_ARG: return "invalid argument";
        case SV_ERR_DTYPE: return "unsupported logit dtype";
        case SV_ERR_SHAPE: return "inconsistent width, row stride or offsets";
        case SV_ERR_LIMIT: return "size above a documented limit";
        case SV_ERR_LAUNCH: return "CUDA launch failed";
        case SV_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
        case SV_ERR_ALIGN: return "pointer not aligned to its element size";
        case SV_ERR_DEVICE: return "no usable CUDA device";
        default: return "unknown status";
    }
}

size_t sv_verify_greedy_workspace(int32_t R, int32_t k, int32_t branches, int32_t V)
{
    if (R < 0 || k < 0 || V < 1 || branches < 1 || branches > SV_MAX_BRANCHES) return 0;
    return greedy_workspace_bytes(R, k, branches, V);
}

int sv_verify_greedy(sv_rows target, int32_t R, int32_t k, int32_t branches, const int32_t* draft,
                     int32_t* accept_len, int32_t* tokens, int32_t* branch, int32_t* status,
                     void* workspace, size_t workspace_bytes, sv_stream_t stream)
{
    if (R < 0 || k < 0) return SV_ERR_INVALID_ARG;
    if (branches < 1 || (branches >= 2 && k < 1)) return SV_ERR_INVALID_ARG;
    if (branches > SV_MAX_BRANCHES) return SV_ERR_LIMIT;
    if (k > SV_MAX_K) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if ((k > 0 && draft == nullptr) || accept_len == nullptr || tokens == nullptr)
        return SV_ERR_INVALID_ARG;
    if (!aligned(draft, 4) || !aligned(accept_len, 4) || !aligned(tokens, 4) ||
        !aligned(branch, 4) || !aligned(status, 4))
        return SV_ERR_ALIGN;
    const int64_t rows = static_cast<int64_t>(R) * (1 + static_cast<int64_t>(branches) * k);
    Rows t{};
    if (int rc = check_rows(target, rows, target.width, &t)) return rc;
    const SegPlan plan = plan_segments(rows, t.width, t.esize);
    if (rows * plan.nseg > INT32_MAX) return SV_ERR_LIMIT;
    if (int rc = check_workspace(workspace, workspace_bytes,
                                 greedy_workspace_bytes(R, k, branches, t.width)))
        return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_verify_greedy(t, R, k, branches, draft, accept_len, tokens, branch,
                                         status, workspace, stream));
}

size_t sv_verify_greedy_top2_workspace(int32_t R, int32_t k, int32_t branches, int32_t V)
{
    if (R < 0 || k < 0 || V < 1 || branches < 1 || branches > SV_MAX_BRANCHES) return 0;
    return greedy_workspace_bytes(R, k, branches, V, true);
}

int sv_verify_greedy_top2(sv_rows target, int32_t R, int32_t k, int32_t branches, const int32_t* draft,
                          int32_t* accept_len, int32_t* tokens, int32_t* branch, int32_t* status,
                          int32_t* top2, void* workspace, size_t workspace_bytes, sv_stream_t stream)
{
    if (R < 0 || k < 0) return SV_ERR_INVALID_ARG;
    if (branches < 1 || (branches >= 2 && k < 1)) return SV_ERR_INVALID_ARG;
    if (branches > SV_MAX_BRANCHES) return SV_ERR_LIMIT;
    if (k > SV_MAX_K) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if ((k > 0 && draft == nullptr) || accept_len == nullptr || tokens == nullptr || top2 == nullptr)
        return SV_ERR_INVALID_ARG;
    if (!aligned(draft, 4) || !aligned(accept_len, 4) || !aligned(tokens, 4) ||
        !aligned(branch, 4) || !aligned(status, 4) || !aligned(top2, 4))
        return SV_ERR_ALIGN;
    const int64_t rows = static_cast<int64_t>(R) * (1 + static_cast<int64_t>(branches) * k);
    Rows t{};
    if (int rc = check_rows(target, rows, target.width, &t)) return rc;
    const SegPlan plan = plan_segments(rows, t.width, t.esize);
    if (rows * plan.nseg > INT32_MAX) return SV_ERR_LIMIT;
    if (int rc = check_workspace(workspace, workspace_bytes,
                                 greedy_workspace_bytes(R, k, branches, t.width, true)))
        return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_verify_greedy(t, R, k, branches, draft, accept_len, tokens, branch,
                                         status, workspace, stream, top2));
}

size_t sv_infer_modality_workspace(int32_t N, int32_t V)
{
    if (N < 0 || V < 1) return 0;
    return modality_workspace_bytes(N, V);
}

int sv_infer_modality(sv_rows logits, int32_t N, const int32_t* part_start, int32_t P, int32_t* amax,
                      int32_t* part, int32_t* mask_lo, int32_t* mask_hi, int32_t* status, void* workspace,
                      size_t workspace_bytes, sv_stream_t stream)
{
    if (N < 0 || P < 1 || part_start == nullptr) return SV_ERR_INVALID_ARG;
    if (P > kMaxParts) return SV_ERR_LIMIT;
    for (int32_t p = 0; p < P; ++p)
        if (part_start[p] > part_start[p + 1]) return SV_ERR_INVALID_ARG;
    if (N == 0) return SV_OK;
    if (part == nullptr) return SV_ERR_INVALID_ARG;
    if (!aligned(amax, 4) || !aligned(part, 4) || !aligned(mask_lo, 4) || !aligned(mask_hi, 4) ||
        !aligned(status, 4))
        return SV_ERR_ALIGN;
    Rows t{};
    if (int rc = check_rows(logits, N, logits.width, &t)) return rc;
    const SegPlan plan = plan_segments(N, t.width, t.esize);
    if (static_cast<int64_t>(N) * plan.nseg > INT32_MAX) return SV_ERR_LIMIT;
    if (int rc = check_workspace(workspace, workspace_bytes, modality_workspace_bytes(N, t.width))) return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    PartTable pt{};
    pt.P = P;
    for (int32_t p = 0; p <= P; ++p) pt.start[p] = part_start[p];
    return launched(launch_infer_modality(t, N, pt, amax, part, mask_lo, mask_hi, status, workspace, stream));
}

size_t sv_verify_sample_workspace(int32_t R, int32_t k, int32_t V, int32_t Vd)
{
    if (R < 0 || k < 0 || V < 1 || Vd < 1) return 0;
    return sample_workspace_bytes(R, k, V, Vd);
}

int sv_verify_sample(sv_rows target, sv_rows draft_logits, const int32_t* d2t, const void* d2t_plan,
                     int32_t R, int32_t k, const int32_t* draft, const uint64_t* seeds,
                     const float* temperature, int32_t* accept_len, int32_t* tokens, float* tv,
                     float* p_draft, float* q_draft, int32_t* status, void* workspace,
                     size_t workspace_bytes, sv_stream_t stream)
{
    if (R < 0 || k < 0) return SV_ERR_INVALID_ARG;
    if (k > SV_MAX_K) return SV_ERR_LIMIT;
    if (static_cast<int64_t>(R) * (k + 1) > INT32_MAX) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if ((k > 0 && draft == nullptr) || seeds == nullptr || temperature == nullptr ||
        accept_len == nullptr || tokens == nullptr)
        return SV_ERR_INVALID_ARG;
    if (!aligned(draft, 4) || !aligned(seeds, 8) || !aligned(temperature, 4) ||
        !aligned(accept_len, 4) || !aligned(tokens, 4) || !aligned(tv, 4) ||
        !aligned(p_draft, 4) || !aligned(q_draft, 4) || !aligned(status, 4) || !aligned(d2t, 4))
        return SV_ERR_ALIGN;
    if (!aligned(d2t_plan, 256)) return SV_ERR_WORKSPACE;
    Rows t{}, d{};
    if (int rc = check_rows(target, static_cast<int64_t>(R) * (k + 1), target.width, &t)) return rc;
    const int64_t drows = static_cast<int64_t>(R) * k;
    if (drows > 0) {
        if (int rc = check_rows(draft_logits, drows, draft_logits.width, &d)) return rc;
    } else {
        d = Rows{nullptr, SV_F32, 4, draft_logits.width > 0 ? draft_logits.width : t.width, 0, false};
    }
    const bool mapped = d2t != nullptr || d2t_plan != nullptr;
    if (!mapped && d.width != t.width) return SV_ERR_SHAPE;
    if (t.width > sample_max_plan_width()) return SV_ERR_LIMIT;  // the race keeps one sum per 2048 ids
    if (int rc = check_workspace(workspace, workspace_bytes,
                                 sample_workspace_bytes(R, k, t.width, d.width)))
        return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_verify_sample(t, d, d2t, d2t_plan, R, k, draft, seeds, temperature, accept_len,
                                         tokens, tv, p_draft, q_draft, status, workspace, stream));
}

size_t sv_d2t_plan_bytes(int32_t V, int32_t Vd)
{
    if (V < 1 || Vd < 1) return 0;
    return d2t_plan_bytes(V, Vd);
}

int sv_d2t_plan_build(const int32_t* d2t, int32_t Vd, int32_t V, void* plan, size_t plan_bytes,
                      sv_stream_t stream)
{
    if (V < 1 || Vd < 1 || d2t == nullptr) return SV_ERR_INVALID_ARG;
    if (V > sample_max_plan_width() || Vd > 65535) return SV_ERR_LIMIT;
    if (!aligned(d2t, 4)) return SV_ERR_ALIGN;
    if (int rc = check_workspace(plan, plan_bytes, d2t_plan_bytes(V, Vd))) return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_d2t_plan_build(d2t, Vd, V, plan, stream));
}

size_t sv_cfg_merge_sample_workspace(int32_t R, int32_t k, int32_t S, int32_t W)
{
    if (R < 0 || k < 0 || S < 1 || S > SV_MAX_S || W < 1) return 0;
    return cfg_workspace_bytes(R, k, S, W);
}

int sv_cfg_merge_sample(sv_rows cond, sv_rows uncond, const int32_t* cb_id_base,
                        const int32_t* cb_data_offset, int32_t S, float w, sv_rows draft_logits,
                        int32_t R, int32_t k, const int32_t* draft, const uint64_t* seeds,
                        const float* temperature, int32_t* accept_len, int32_t* tokens, float* tv,
                        int32_t* status, void* workspace, size_t workspace_bytes,
                        sv_stream_t stream)
{
    if (R < 0 || k < 0 || S < 1) return SV_ERR_INVALID_ARG;
    if (k > SV_MAX_K || S > SV_MAX_S) return SV_ERR_LIMIT;
    if (cb_id_base == nullptr) return SV_ERR_INVALID_ARG;
    if (cond.width > cfg_max_width()) return SV_ERR_LIMIT;
    if (cond.width != uncond.width || cond.dtype != uncond.dtype ||
        cond.row_stride != uncond.row_stride)
        return SV_ERR_SHAPE;
    if (R == 0) return SV_OK;
    if ((k > 0 && draft == nullptr) || seeds == nullptr || temperature == nullptr ||
        accept_len == nullptr || tokens == nullptr)
        return SV_ERR_INVALID_ARG;
    if (!aligned(draft, 4) || !aligned(seeds, 8) || !aligned(temperature, 4) ||
        !aligned(accept_len, 4) || !aligned(tokens, 4) || !aligned(tv, 4) || !aligned(status, 4))
        return SV_ERR_ALIGN;
    CfgShape shape{};
    shape.S = S;
    shape.W = cond.width;
    shape.w = w;
    int64_t max_end = cond.width;
    for (int s = 0; s < S; ++s) {
        shape.id_base[s] = cb_id_base[s];
        shape.data_off[s] = cb_data_offset ? cb_data_offset[s] : 0;
        if (shape.data_off[s] < 0) return SV_ERR_SHAPE;
        max_end = std::max<int64_t>(max_end, static_cast<int64_t>(shape.data_off[s]) + cond.width);
    }
    const int64_t rows = static_cast<int64_t>(R) * (k + 1) * S;
    Rows c{}, u{}, d{};
    if (int rc = check_rows(cond, rows, max_end, &c)) return rc;
    if (int rc = check_rows(uncond, rows, max_end, &u)) return rc;
    const Rows* dp = nullptr;
    if (draft_logits.data != nullptr && k > 0) {
        if (draft_logits.width != cond.width) return SV_ERR_SHAPE;
        if (int rc = check_rows(draft_logits, static_cast<int64_t>(R) * k * S, draft_logits.width, &d))
            return rc;
        dp = &d;
    }
    if (int rc = check_workspace(workspace, workspace_bytes, cfg_workspace_bytes(R, k, S, cond.width)))
        return rc;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_cfg_merge_sample(c, u, shape, dp, R, k, draft, seeds, temperature,
                                            accept_len, tokens, tv, status, workspace, stream));
}

int sv_pool_append(int32_t* pool, int32_t* pool_len, int32_t Lp, const int32_t* drafts, int32_t k,
                   int32_t R, int32_t* status, sv_stream_t stream)
{
    if (R < 0 || k < 0 || Lp < 0) return SV_ERR_INVALID_ARG;
    if (k > SV_MAX_K || Lp > SV_MAX_POOL) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if (pool_len == nullptr || (k > 0 && drafts == nullptr) || (Lp > 0 && pool == nullptr))
        return SV_ERR_INVALID_ARG;
    if (!aligned(pool, 4) || !aligned(pool_len, 4) || !aligned(drafts, 4) || !aligned(status, 4))
        return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_pool_append(pool, pool_len, Lp, drafts, k, R, status, stream));
}

int sv_pool_lookup(const int32_t* pool, const int32_t* pool_len, int32_t Lp, const int32_t* suffix,
                   int32_t N, int32_t R, int32_t gamma, int32_t* match_len, int32_t* cont,
                   sv_stream_t stream)
{
    if (R < 0 || N < 0 || gamma < 0 || Lp < 0) return SV_ERR_INVALID_ARG;
    if (N > SV_MAX_NGRAM || gamma > SV_MAX_K || Lp > SV_MAX_POOL) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if (pool_len == nullptr || match_len == nullptr || (Lp > 0 && pool == nullptr) ||
        (N > 0 && suffix == nullptr) || (gamma > 0 && cont == nullptr))
        return SV_ERR_INVALID_ARG;
    if (!aligned(pool, 4) || !aligned(pool_len, 4) || !aligned(suffix, 4) || !aligned(match_len, 4) ||
        !aligned(cont, 4))
        return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_pool_lookup(pool, pool_len, Lp, suffix, N, R, gamma, match_len, cont, stream));
}

int sv_suffix_append(int32_t* suffix, int32_t N, int32_t R, const int32_t* tokens, const int32_t* accept_len,
                     int32_t k, sv_stream_t stream)
{
    if (R < 0 || N < 0 || k < 0) return SV_ERR_INVALID_ARG;
    if (N > SV_MAX_NGRAM || k > SV_MAX_K) return SV_ERR_LIMIT;
    if (R == 0 || N == 0) return SV_OK;
    if (suffix == nullptr || tokens == nullptr || accept_len == nullptr) return SV_ERR_INVALID_ARG;
    if (!aligned(suffix, 4) || !aligned(tokens, 4) || !aligned(accept_len, 4)) return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_suffix_append(suffix, N, R, tokens, accept_len, k, stream));
}

int sv_accept_scan(const uint8_t* accept, const int32_t* draft, const int32_t* fix, int32_t R,
                   int32_t k, int32_t* accept_len, int32_t* tokens, sv_stream_t stream)
{
    if (R < 0 || k < 0) return SV_ERR_INVALID_ARG;
    if (k > SV_MAX_K) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if ((k > 0 && (accept == nullptr || draft == nullptr)) || fix == nullptr ||
        accept_len == nullptr || tokens == nullptr)
        return SV_ERR_INVALID_ARG;
    if (!aligned(draft, 4) || !aligned(fix, 4) || !aligned(accept_len, 4) || !aligned(tokens, 4))
        return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_accept_scan(accept, draft, fix, R, k, accept_len, tokens, stream));
}

int sv_step_tables(const int32_t* seq_len, const int32_t* new_len, int32_t R, int32_t block_size,
                   int32_t* block_table, int32_t max_blocks, const int32_t* free_blocks,
                   const int32_t* free_count, int32_t num_blocks, const int32_t* parent, int32_t T,
                   int32_t* cu_tokens, int32_t* kv_len, int64_t* slot, int32_t* position, uint32_t* mask,
                   int32_t mask_words, int32_t* free_count_out, int32_t* status, sv_stream_t stream)
{
    if (R < 0 || T < 0 || block_size < 1 || max_blocks < 0 || num_blocks < 0) return SV_ERR_INVALID_ARG;
    if (mask_words < 0 || (parent != nullptr && mask_words < 1)) return SV_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks) * block_size > INT32_MAX) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if (seq_len == nullptr || new_len == nullptr || free_count == nullptr || cu_tokens == nullptr ||
        kv_len == nullptr || free_count_out == nullptr || (max_blocks > 0 && block_table == nullptr) ||
        (num_blocks > 0 && free_blocks == nullptr))
        return SV_ERR_INVALID_ARG;
    if (T > 0 && (slot == nullptr || position == nullptr || (parent != nullptr && mask == nullptr)))
        return SV_ERR_INVALID_ARG;
    if (!aligned(seq_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
        !aligned(free_count, 4) || !aligned(parent, 4) || !aligned(cu_tokens, 4) || !aligned(kv_len, 4) ||
        !aligned(slot, 8) || !aligned(position, 4) || !aligned(mask, 4) || !aligned(free_count_out, 4) ||
        !aligned(status, 4))
        return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    const StepTablesArgs a{seq_len,     new_len,    R,      block_size, max_blocks, num_blocks, T,
                           mask_words,  divisor_of(block_size), block_table, free_blocks, free_count, parent, cu_tokens, kv_len,
                           slot,        position,   mask,   free_count_out, status};
    return launched(launch_step_tables(a, stream));
}

int sv_rope_cache(sv_heads q, sv_heads k, sv_heads v, const int32_t* position, const int64_t* slot,
                  const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, float mscale, sv_heads q_out,
                  sv_kv_cache cache, sv_stream_t stream)
{
    if (interleaved != 0 && interleaved != 1) return SV_ERR_INVALID_ARG;
    if (q.tokens < 0) return SV_ERR_INVALID_ARG;
    if (int rc = check_cache(cache, q.tokens > 0)) return rc;
    if (cache.layers != 1) return SV_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > cache.head_dim) return SV_ERR_SHAPE;
    if (q.tokens == 0) return SV_OK;
    if (int rc = check_heads(q, cache.dtype, cache.head_dim, q.tokens)) return rc;
    if (int rc = check_heads(k, cache.dtype, cache.head_dim, q.tokens)) return rc;
    if (int rc = check_heads(v, cache.dtype, cache.head_dim, q.tokens)) return rc;
    if (int rc = check_heads(q_out, cache.dtype, cache.head_dim, q.tokens)) return rc;
    if (k.heads != cache.kv_heads || v.heads != cache.kv_heads || q_out.heads != q.heads) return SV_ERR_SHAPE;
    if (static_cast<int64_t>(q.heads) + 2 * static_cast<int64_t>(cache.kv_heads) > 65536) return SV_ERR_LIMIT;
    if (position == nullptr || slot == nullptr || (rot_dim > 0 && freqs == nullptr)) return SV_ERR_INVALID_ARG;
    if (!aligned(position, 4) || !aligned(slot, 8) || !aligned(freqs, 8)) return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_rope_cache(RopeArgs{q, k, v, q_out, position, slot, freqs, rot_dim, interleaved,
                                               mscale, cache},
                                      stream));
}

int sv_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double trained, double low,
                  double high, uint64_t* freqs)
{
    if (rot_dim < 0 || rot_dim % 2 != 0 || !(base > 0.0) || !std::isfinite(base)) return SV_ERR_INVALID_ARG;
    if (scaling < SV_ROPE_PLAIN || scaling > SV_ROPE_BY_TURNS) return SV_ERR_INVALID_ARG;
    if (scaling != SV_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return SV_ERR_INVALID_ARG;
    if (scaling == SV_ROPE_BASE && rot_dim == 2) return SV_ERR_SHAPE;  // its exponent has no value there
    const bool parts = scaling == SV_ROPE_BY_DIM || scaling == SV_ROPE_BY_TURNS;
    if (parts && (!(trained > 0.0) || !(low > 0.0) || !(high > low) || !std::isfinite(trained) || !std::isfinite(high)))
        return SV_ERR_INVALID_ARG;
    if (scaling == SV_ROPE_BY_DIM && !(base > 1.0)) return SV_ERR_INVALID_ARG;
    if (rot_dim == 0) return SV_OK;
    if (freqs == nullptr) return SV_ERR_INVALID_ARG;
    if (!aligned(freqs, 8)) return SV_ERR_ALIGN;
    const double two_pi = 6.283185307179586476925286766559;
    const int32_t half = rot_dim / 2;
    const double b = scaling == SV_ROPE_BASE ? base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2)) : base;
    // the pair index (not rounded) whose frequency turns `t` times within the trained positions
    auto index_of = [&](double t) { return half * std::log(trained / (t * two_pi)) / std::log(base); };
    for (int32_t i = 0; i < half; ++i) {
        double f = std::pow(b, -static_cast<double>(i) / half);
        if (scaling == SV_ROPE_LINEAR) f /= factor;
        if (parts) {
            double keep;  // 1: the frequency stays, 0: stretched by the factor
            if (scaling == SV_ROPE_BY_TURNS) {
                keep = (trained * f / two_pi - low) / (high - low);
            } else {
                const double first = std::max(0.0, std::floor(index_of(high)));
                const double last = std::min(static_cast<double>(rot_dim - 1), std::ceil(index_of(low)));
                keep = 1.0 - (i - first) / std::max(last - first, 1e-3);
            }
            keep = std::min(1.0, std::max(0.0, keep));
            f = f / factor * (1.0 - keep) + f * keep;
        }
        // whole turns per position drop out; 2^64 itself would be a whole turn
        double turns = f / two_pi;
        turns -= std::floor(turns);
        const double scaled = std::nearbyint(turns * 18446744073709551616.0);
        freqs[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
    }
    return SV_OK;
}

size_t sv_tree_attention_workspace(int32_t R, int32_t T, int32_t max_tokens, int32_t heads, int32_t kv_heads,
                                   int32_t head_dim, int64_t max_kv)
{
    if (R < 0 || T < 0 || max_tokens < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || head_dim < 1 ||
        head_dim > SV_MAX_HEAD_DIM || max_kv < 0 || max_kv > INT32_MAX || heads / kv_heads > SV_MAX_GROUP)
        return 0;
    return attn_workspace_bytes(R, max_tokens, heads, kv_heads, head_dim, max_kv);
}

int sv_tree_attention(sv_heads q, sv_kv_cache cache, const int32_t* block_table, int32_t max_blocks,
                      const int32_t* kv_len, const int32_t* cu_tokens, int32_t R, int32_t max_tokens,
                      const uint32_t* mask, int32_t mask_words, float scale, sv_heads out, float* lse,
                      int32_t* status, void* workspace, size_t workspace_bytes, sv_stream_t stream)
{
    return tree_attention(AttnArgs{q, out, cache, block_table, max_blocks, kv_len, cu_tokens, R, max_tokens, mask,
                                   mask_words, scale, lse, status, workspace, -1},
                          workspace_bytes, stream);
}

int sv_selftest_tree_attention_stop(sv_heads q, sv_kv_cache cache, const int32_t* block_table, int32_t max_blocks,
                                    const int32_t* kv_len, const int32_t* cu_tokens, int32_t R, int32_t max_tokens,
                                    const uint32_t* mask, int32_t mask_words, float scale, sv_heads out, float* lse,
                                    int32_t* status, void* workspace, size_t workspace_bytes, int32_t cta,
                                    sv_stream_t stream)
{
    if (cta < 0) return SV_ERR_INVALID_ARG;
    return tree_attention(AttnArgs{q, out, cache, block_table, max_blocks, kv_len, cu_tokens, R, max_tokens, mask,
                                   mask_words, scale, lse, status, workspace, cta},
                          workspace_bytes, stream);
}

int sv_cache_commit(sv_kv_cache cache, const int32_t* block_table, int32_t max_blocks, const int32_t* seq_len,
                    const int32_t* kv_len, const int32_t* cu_tokens, int32_t R, const int32_t* accept_len,
                    const int32_t* branch, const int32_t* path, int32_t k, int32_t* free_blocks,
                    const int32_t* free_count, int32_t* seq_len_out, int32_t* free_count_out, int32_t* status,
                    sv_stream_t stream)
{
    if (R < 0 || k < 0 || max_blocks < 0) return SV_ERR_INVALID_ARG;
    if (k > SV_MAX_K) return SV_ERR_LIMIT;
    if (branch != nullptr && path != nullptr) return SV_ERR_INVALID_ARG;
    if (int rc = check_cache(cache, R > 0)) return rc;
    // 128 16-byte columns of the heads to a row of the launch grid
    if (2ll * cache.layers * cache.kv_heads * (cache.head_dim / 8) > 65535ll * 128) return SV_ERR_LIMIT;
    if (static_cast<int64_t>(max_blocks) * cache.block_size > INT32_MAX) return SV_ERR_LIMIT;
    if (R == 0) return SV_OK;
    if (seq_len == nullptr || kv_len == nullptr || cu_tokens == nullptr || accept_len == nullptr ||
        free_blocks == nullptr || free_count == nullptr || seq_len_out == nullptr || free_count_out == nullptr ||
        (max_blocks > 0 && block_table == nullptr))
        return SV_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(seq_len, 4) || !aligned(kv_len, 4) || !aligned(cu_tokens, 4) ||
        !aligned(accept_len, 4) || !aligned(branch, 4) || !aligned(path, 4) || !aligned(free_blocks, 4) ||
        !aligned(free_count, 4) || !aligned(seq_len_out, 4) || !aligned(free_count_out, 4) || !aligned(status, 4))
        return SV_ERR_ALIGN;
    if (!have_device()) return SV_ERR_DEVICE;
    return launched(launch_cache_commit(CommitArgs{cache, block_table, max_blocks, seq_len, kv_len, cu_tokens, R,
                                                   accept_len, branch, path, k, divisor_of(cache.block_size),
                                                   free_blocks, free_count, seq_len_out, free_count_out, status},
                                        stream));
}

}  // extern "C"
