// csa_api.cu -- the C ABI declared in include/csa.h: host-side argument checks,
// workspace sizing and kernel dispatch. Nothing here allocates memory; every
// call only enqueues work on the caller's stream.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "common.cuh"

namespace csa {
cudaError_t launch_compress(const csa_cache &c, const void *kv_tok, const void *idx_tok, const float *gate_w,
                            const int32_t *tok_offsets, int32_t n_tokens, cudaStream_t s);
size_t index_topk_workspace_bytes(const csa_cache &c, int Nq);
size_t index_topk_min_workspace_bytes(const csa_cache &c, int Nq, int H_I);
cudaError_t launch_index_topk(const csa_cache &c, const void *q_idx, const float *w, int Nq, int H_I,
                              const int32_t *q_offsets, const int32_t *q_pos, int topk, int32_t *sel_idx,
                              void *workspace, size_t workspace_bytes, int num_sms, cudaStream_t s);
size_t index_pool_workspace_bytes(int Nq, int cap, int G, int P);
cudaError_t launch_index_topk_pool(const csa_cache &c, const void *q_idx, const float *w, int Nq, int H_I,
                                   const int32_t *q_offsets, const int32_t *q_pos, int topk, int32_t *sel_idx,
                                   int pool_shift, int P, int32_t *pool_blk, void *workspace, int num_sms,
                                   cudaStream_t s);
size_t index_reindex_workspace_bytes(int Nq, int G, int P);
cudaError_t launch_index_topk_reindex(const csa_cache &c, const void *q_idx, const float *w, int Nq, int H_I,
                                      const int32_t *q_offsets, const int32_t *q_pos, int topk, int32_t *sel_idx,
                                      int pool_shift, int P, const int32_t *pool_blk, void *workspace, int num_sms,
                                      cudaStream_t s, int layers);
size_t attend_workspace_bytes(int Nq, int D, int num_ctas);
cudaError_t launch_mxf4_probe(int iters, int32_t *status, int num_sms, cudaStream_t s);
cudaError_t launch_attend(const csa_cache &c, const void *q, int Nq, int H, const int32_t *q_offsets,
                          const int32_t *q_pos, const int32_t *sel_idx, int topk, const void *win_kv,
                          const int64_t *win_start, const int32_t *win_len, int max_win, float softmax_scale,
                          float *out, float *lse, void *workspace, int num_ctas, cudaStream_t s);
size_t shared_attend_workspace_bytes(int batch, int Nq, int H, int D, int num_sms);
cudaError_t launch_shared_attend(const csa_cache &c, const void *q, int Nq, int H, const int32_t *q_offsets,
                                 const int32_t *q_pos, const float *join_out, const float *join_lse,
                                 float softmax_scale, void *out, float *lse, void *workspace, int num_sms,
                                 cudaStream_t s);
size_t cache_copy_workspace_bytes(int dst_batch, int jobs, int cols);
cudaError_t launch_cache_copy(const csa_cache &src, const csa_cache &dst, int jobs, const int32_t *src_slot,
                              const int32_t *dst_slot, const int32_t *keep, int cols, const int32_t *max_blocks,
                              void *workspace, int num_sms, cudaStream_t s);
cudaError_t launch_rotary(const csa_vectors &x, const csa_vectors &out, int rows, int heads, int dim,
                          const csa_rope &rope, const int32_t *pos, bool inverse, bool in_place, cudaStream_t s);
}  // namespace csa

namespace {

constexpr int kMaxCapacity = 1 << 19;  // the top-k select keeps two bitmaps of this many bits in shared memory
constexpr int kMaxTopk = 4096;
constexpr int kMaxReindexLayers = 16;  // Reindex layers in one csa_index_topk_reindex_layers call

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Number of SMs of the current device (the attention and scan grids are sized from it).
int num_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

csa_status check_cache(const csa_cache *c) {
    if (!c || !c->fp4 || !c->scale || !c->n_blocks) return CSA_ERR_NULL;
    if (c->batch < 1 || c->capacity < 1 || c->block < 1 || c->block > 128) return CSA_ERR_SHAPE;
    if (c->dim < 64 || c->dim % 32 != 0) return CSA_ERR_SHAPE;
    if (c->capacity > kMaxCapacity) return CSA_ERR_UNSUPPORTED;
    if (c->scale_fmt != CSA_SCALE_E8M0_32 && c->scale_fmt != CSA_SCALE_E4M3_16) return CSA_ERR_SHAPE;
    if (!aligned(c->fp4, 16) || !aligned(c->scale, 16) || !aligned(c->n_blocks, 4)) return CSA_ERR_ALIGN;
    if (c->status && !aligned(c->status, 4)) return CSA_ERR_ALIGN;
    if (c->idx_key) {
        if (c->idx_dtype != CSA_IDX_BF16 && c->idx_dtype != CSA_IDX_E4M3 && c->idx_dtype != CSA_IDX_MXFP4)
            return CSA_ERR_SHAPE;
        if (c->idx_dim != 64 && c->idx_dim != 128 && c->idx_dim != 256) return CSA_ERR_UNSUPPORTED;
        if (!aligned(c->idx_key, 16)) return CSA_ERR_ALIGN;
        if (c->idx_dtype == CSA_IDX_MXFP4) {
            if (!c->idx_key_scale) return CSA_ERR_NULL;
            if (!aligned(c->idx_key_scale, 4)) return CSA_ERR_ALIGN;
        }
    }
    return CSA_OK;
}

// ---- slot copies (csa_cache_copy)
constexpr int kMaxCopyDim = 512;
constexpr int kMaxCopyJobs = 65535;  // a grid dimension

int64_t scale_row(const csa_cache &c) { return c.dim / (c.scale_fmt == CSA_SCALE_E4M3_16 ? 16 : 32); }
int64_t key_row(const csa_cache &c) {
    return c.idx_dtype == CSA_IDX_BF16 ? 2 * c.idx_dim : c.idx_dtype == CSA_IDX_E4M3 ? c.idx_dim : c.idx_dim / 2;
}
bool ranges_meet(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
// One cache with itself, or two that share nothing.
bool same_or_apart(const csa_cache &a, const csa_cache &b) {
    if (a.fp4 == b.fp4 && a.scale == b.scale && a.idx_key == b.idx_key && a.idx_key_scale == b.idx_key_scale &&
        a.n_blocks == b.n_blocks && a.batch == b.batch && a.capacity == b.capacity)
        return true;
    const int64_t na = (int64_t)a.batch * a.capacity, nb = (int64_t)b.batch * b.capacity;
    return !ranges_meet(a.fp4, na * (a.dim / 2), b.fp4, nb * (b.dim / 2)) &&
           !ranges_meet(a.scale, na * scale_row(a), b.scale, nb * scale_row(b)) &&
           !ranges_meet(a.idx_key, na * key_row(a), b.idx_key, nb * key_row(b)) &&
           !ranges_meet(a.idx_key_scale, na * (a.idx_dim / 32), b.idx_key_scale, nb * (b.idx_dim / 32)) &&
           !ranges_meet(a.n_blocks, 4 * (int64_t)a.batch, b.n_blocks, 4 * (int64_t)b.batch);
}

// ---- strided vectors (csa_rotary)
constexpr int kMaxRotaryDim = 8192;

struct VectorShape {
    int64_t rows, heads, dim;
};

bool dtype_ok(int32_t t) { return t == CSA_BF16 || t == CSA_F32; }
int dtype_size(int32_t t) { return t == CSA_BF16 ? 2 : 4; }

// No negative strides, and no byte offset beyond 2^62 (nothing below can then wrap).
bool strides_ok(const csa_vectors &v, const VectorShape &n) {
    constexpr int64_t kMost = int64_t(1) << 60;
    if (v.row_stride < 0 || v.head_stride < 0) return false;
    if (n.rows > 1 && v.row_stride > kMost / n.rows) return false;
    if (n.heads > 1 && v.head_stride > kMost / n.heads) return false;
    return true;
}
int64_t row_step(const csa_vectors &v, const VectorShape &n) { return n.rows > 1 ? v.row_stride : 0; }
int64_t head_step(const csa_vectors &v, const VectorShape &n) { return n.heads > 1 ? v.head_stride : 0; }

bool same_layout(const csa_vectors &a, const csa_vectors &b, const VectorShape &n) {
    return a.dtype == b.dtype && row_step(a, n) == row_step(b, n) && head_step(a, n) == head_step(b, n);
}

// Whether some offset row * rs + head * hs (not 0, 0 when `apart`) lies within dim of `delta`:
// then two vectors share a channel. Checked over the axis with fewer steps.
bool meets(int64_t delta, int64_t rs, int64_t hs, const VectorShape &n, bool apart) {
    int64_t few = n.heads, many = n.rows, fs = hs, ms = rs;
    if (n.rows < n.heads) {
        few = n.rows, many = n.heads, fs = rs, ms = hs;
    }
    for (int64_t f = -(few - 1); f < few; ++f) {
        const int64_t rest = delta - f * fs;  // look for m with |rest - m * ms| < dim, |m| < many
        int64_t m = ms > 0 ? rest / ms : 0;
        for (int64_t k = m - 1; k <= m + 1; ++k) {
            if (k <= -many || k >= many || (apart && f == 0 && k == 0)) continue;
            const int64_t d = rest - k * ms;
            if (d < n.dim && -d < n.dim) return true;
        }
    }
    return false;
}
bool self_overlap(const csa_vectors &v, const VectorShape &n) {
    const int64_t rs = row_step(v, n), hs = head_step(v, n);
    if ((n.heads == 1 || hs >= n.dim) && (n.rows == 1 || rs >= (n.heads - 1) * hs + n.dim)) return false;
    return meets(0, row_step(v, n), head_step(v, n), n, true);
}
// Whether two tensors of the same shape share memory: with the same strides and type exactly,
// otherwise by their ranges.
bool overlap(const csa_vectors &a, const csa_vectors &b, const VectorShape &n) {
    auto span = [&](const csa_vectors &v) {
        return ((n.rows - 1) * row_step(v, n) + (n.heads - 1) * head_step(v, n) + n.dim) * dtype_size(v.dtype);
    };
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
    if (pa + (uintptr_t)span(a) <= pb || pb + (uintptr_t)span(b) <= pa) return false;
    const int64_t bytes = (int64_t)pb - (int64_t)pa;
    if (!same_layout(a, b, n) || bytes % dtype_size(a.dtype) != 0) return true;
    return meets(bytes / dtype_size(a.dtype), row_step(a, n), head_step(a, n), n, false);
}

csa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

}  // namespace

// Argument checks of every indexer call (csa_index_topk, its pool and Reindex
// forms, and csa_index_topk_noalloc in noalloc.cu), in the order the status
// codes are reported; the workspace is checked by each caller afterwards.
namespace csa {
csa_status check_index_args(const csa_cache *cache, const void *q_idx, const float *w, int32_t n_queries,
                            int32_t idx_heads, const int32_t *q_offsets, const int32_t *q_pos, int32_t topk,
                            const int32_t *sel_idx) {
    csa_status st = check_cache(cache);
    if (st != CSA_OK) return st;
    if (!cache->idx_key || !q_idx || !w || !q_offsets || !q_pos || !sel_idx) return CSA_ERR_NULL;
    if (n_queries < 1 || idx_heads < 1 || topk < 1) return CSA_ERR_SHAPE;
    if (idx_heads > 8 || topk > kMaxTopk) return CSA_ERR_UNSUPPORTED;
    if (cache->idx_dtype == CSA_IDX_MXFP4 && idx_heads > 4) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q_idx, 16) || !aligned(w, 4) || !aligned(q_offsets, 4) || !aligned(q_pos, 4) ||
        !aligned(sel_idx, 4))
        return CSA_ERR_ALIGN;
    return CSA_OK;
}
}  // namespace csa

extern "C" {

const char *csa_status_string(int32_t status) {
    switch (status) {
        case CSA_OK: return "ok";
        case CSA_ERR_NULL: return "required pointer is NULL";
        case CSA_ERR_SHAPE: return "size out of range or inconsistent";
        case CSA_ERR_ALIGN: return "pointer not aligned";
        case CSA_ERR_UNSUPPORTED: return "configuration not implemented";
        case CSA_ERR_WORKSPACE: return "workspace missing or too small";
        case CSA_ERR_CUDA: return "CUDA runtime error";
        default: return "unknown status";
    }
}

int32_t csa_version(void) { return 103; }

csa_status csa_compress_quantize(const csa_cache *cache, const void *kv_tok, const void *idx_tok, const float *gate_w,
                                 const int32_t *tok_offsets, int32_t n_tokens, csa_stream_t stream) {
    csa_status st = check_cache(cache);
    if (st != CSA_OK) return st;
    if (!kv_tok || !gate_w || !tok_offsets) return CSA_ERR_NULL;
    if ((cache->idx_key != nullptr) != (idx_tok != nullptr)) return CSA_ERR_NULL;
    if (n_tokens < 0) return CSA_ERR_SHAPE;
    if (cache->dim != 64 && cache->dim != 128 && cache->dim != 256 && cache->dim != 512) return CSA_ERR_UNSUPPORTED;
    if (!aligned(kv_tok, 16) || !aligned(gate_w, 16) || !aligned(tok_offsets, 4)) return CSA_ERR_ALIGN;
    if (idx_tok && !aligned(idx_tok, 16)) return CSA_ERR_ALIGN;
    return from_cuda(csa::launch_compress(*cache, kv_tok, idx_tok, gate_w, tok_offsets, n_tokens,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t csa_index_topk_workspace(const csa_cache *cache, int32_t n_queries, int32_t topk) {
    if (!cache || n_queries < 1 || topk < 1 || cache->capacity < 1 || cache->capacity > kMaxCapacity) return 0;
    return csa::index_topk_workspace_bytes(*cache, n_queries);
}

csa_status csa_index_topk(const csa_cache *cache, const void *q_idx, const float *w, int32_t n_queries,
                          int32_t idx_heads, const int32_t *q_offsets, const int32_t *q_pos, int32_t topk,
                          int32_t *sel_idx, void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    const csa_status st = csa::check_index_args(cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk,
                                                 sel_idx);
    if (st != CSA_OK) return st;
    // one chunk of queries must fit; a larger workspace runs more queries per chunk
    const size_t need = csa::index_topk_min_workspace_bytes(*cache, n_queries, idx_heads);
    if (!workspace || workspace_bytes < need) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return CSA_ERR_CUDA;
    return from_cuda(csa::launch_index_topk(*cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk, sel_idx,
                                            workspace, workspace_bytes, sms, reinterpret_cast<cudaStream_t>(stream)));
}

// log2 of a pool block size (1, 2, 4, ... 32 entries), or -1
static int pool_shift_of(int32_t g) {
    for (int k = 0; k <= 5; ++k)
        if (g == (1 << k)) return k;
    return -1;
}


static bool pool_sizes_ok(int32_t pool_group, int32_t pool_blocks) {
    return pool_shift_of(pool_group) >= 0 && pool_blocks >= 1 && pool_blocks <= kMaxTopk &&
           (long long)pool_group * pool_blocks <= kMaxCapacity;
}

size_t csa_index_pool_workspace(const csa_cache *cache, int32_t n_queries, int32_t topk, int32_t pool_group,
                                int32_t pool_blocks) {
    if (!cache || n_queries < 1 || topk < 1 || cache->capacity < 1 || cache->capacity > kMaxCapacity ||
        !pool_sizes_ok(pool_group, pool_blocks))
        return 0;
    return csa::index_pool_workspace_bytes(n_queries, cache->capacity, pool_group, pool_blocks);
}

csa_status csa_index_topk_pool(const csa_cache *cache, const void *q_idx, const float *w, int32_t n_queries,
                               int32_t idx_heads, const int32_t *q_offsets, const int32_t *q_pos, int32_t topk,
                               int32_t *sel_idx, int32_t pool_group, int32_t pool_blocks, int32_t *pool_blk,
                               void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    csa_status st = csa::check_index_args(cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk, sel_idx);
    if (st != CSA_OK) return st;
    if (!pool_blk) return CSA_ERR_NULL;
    if (pool_shift_of(pool_group) < 0 || pool_blocks < 1) return CSA_ERR_SHAPE;
    if (!pool_sizes_ok(pool_group, pool_blocks)) return CSA_ERR_UNSUPPORTED;
    if (!aligned(pool_blk, 4)) return CSA_ERR_ALIGN;
    const size_t need = csa_index_pool_workspace(cache, n_queries, topk, pool_group, pool_blocks);
    if (!workspace || workspace_bytes < need) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return CSA_ERR_CUDA;
    return from_cuda(csa::launch_index_topk_pool(*cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk,
                                                 sel_idx, pool_shift_of(pool_group), pool_blocks, pool_blk, workspace,
                                                 sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t csa_index_reindex_layers_workspace(const csa_cache *cache, int32_t n_queries, int32_t n_layers,
                                          int32_t pool_group, int32_t pool_blocks) {
    if (!cache || n_queries < 1 || n_layers < 1 || n_layers > kMaxReindexLayers ||
        !pool_sizes_ok(pool_group, pool_blocks) || (long long)n_queries * n_layers > (1 << 30))
        return 0;
    return csa::index_reindex_workspace_bytes(n_queries * n_layers, pool_group, pool_blocks);
}

size_t csa_index_reindex_workspace(const csa_cache *cache, int32_t n_queries, int32_t pool_group,
                                   int32_t pool_blocks) {
    return csa_index_reindex_layers_workspace(cache, n_queries, 1, pool_group, pool_blocks);
}

csa_status csa_index_topk_reindex_layers(const csa_cache *cache, const void *q_idx, const float *w,
                                         int32_t n_queries, int32_t n_layers, int32_t idx_heads,
                                         const int32_t *q_offsets, const int32_t *q_pos, int32_t topk,
                                         int32_t *sel_idx, int32_t pool_group, int32_t pool_blocks,
                                         const int32_t *pool_blk, void *workspace, size_t workspace_bytes,
                                         csa_stream_t stream) {
    csa_status st = csa::check_index_args(cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk, sel_idx);
    if (st != CSA_OK) return st;
    if (!pool_blk) return CSA_ERR_NULL;
    if (n_layers < 1 || pool_shift_of(pool_group) < 0 || pool_blocks < 1) return CSA_ERR_SHAPE;
    if (n_layers > kMaxReindexLayers || !pool_sizes_ok(pool_group, pool_blocks)) return CSA_ERR_UNSUPPORTED;
    if (!aligned(pool_blk, 4)) return CSA_ERR_ALIGN;
    const size_t need = csa_index_reindex_layers_workspace(cache, n_queries, n_layers, pool_group, pool_blocks);
    if (!workspace || workspace_bytes < need) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return CSA_ERR_CUDA;
    return from_cuda(csa::launch_index_topk_reindex(*cache, q_idx, w, n_queries, idx_heads, q_offsets, q_pos, topk,
                                                    sel_idx, pool_shift_of(pool_group), pool_blocks, pool_blk,
                                                    workspace, sms, reinterpret_cast<cudaStream_t>(stream),
                                                    n_layers));
}

csa_status csa_index_topk_reindex(const csa_cache *cache, const void *q_idx, const float *w, int32_t n_queries,
                                  int32_t idx_heads, const int32_t *q_offsets, const int32_t *q_pos, int32_t topk,
                                  int32_t *sel_idx, int32_t pool_group, int32_t pool_blocks,
                                  const int32_t *pool_blk, void *workspace, size_t workspace_bytes,
                                  csa_stream_t stream) {
    return csa_index_topk_reindex_layers(cache, q_idx, w, n_queries, 1, idx_heads, q_offsets, q_pos, topk, sel_idx,
                                         pool_group, pool_blocks, pool_blk, workspace, workspace_bytes, stream);
}

size_t csa_attend_workspace(const csa_cache *cache, int32_t n_queries, int32_t heads) {
    if (!cache || n_queries < 1 || heads < 1 || (cache->dim != 128 && cache->dim != 512)) return 0;
    const int sms = num_sms();
    if (sms <= 0) return 0;
    return csa::attend_workspace_bytes(n_queries, cache->dim, sms);
}

static csa_status check_attend(const csa_cache *cache, const void *q, int32_t n_queries, int32_t heads,
                               const int32_t *q_offsets, const void *win_kv, const int64_t *win_start,
                               const int32_t *win_len, int32_t max_win, float *out, float *lse, void *workspace,
                               size_t workspace_bytes) {
    csa_status st = check_cache(cache);
    if (st != CSA_OK) return st;
    if (!q || !q_offsets || !out) return CSA_ERR_NULL;
    const bool any_win = win_kv || win_start || win_len;
    if (any_win && !(win_kv && win_start && win_len)) return CSA_ERR_NULL;
    if (n_queries < 1 || heads < 1 || max_win < 0) return CSA_ERR_SHAPE;
    if (heads > 64 || (cache->dim != 128 && cache->dim != 512)) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(q_offsets, 4) || !aligned(out, 16)) return CSA_ERR_ALIGN;
    if (lse && !aligned(lse, 4)) return CSA_ERR_ALIGN;
    if (any_win && (!aligned(win_kv, 16) || !aligned(win_start, 8) || !aligned(win_len, 4))) return CSA_ERR_ALIGN;
    const size_t need = csa_attend_workspace(cache, n_queries, heads);
    if (need == 0) return CSA_ERR_CUDA;
    if (!workspace || workspace_bytes < need) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    return CSA_OK;
}

csa_status csa_decode_attend(const csa_cache *cache, const void *q, int32_t n_queries, int32_t heads,
                             const int32_t *q_offsets, const int32_t *sel_idx, int32_t topk, const void *win_kv,
                             const int64_t *win_start, const int32_t *win_len, int32_t max_win, float softmax_scale,
                             float *out, float *lse, void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    csa_status st = check_attend(cache, q, n_queries, heads, q_offsets, win_kv, win_start, win_len, max_win, out, lse,
                                 workspace, workspace_bytes);
    if (st != CSA_OK) return st;
    if (!sel_idx) return CSA_ERR_NULL;
    if (topk < 1) return CSA_ERR_SHAPE;
    if (!aligned(sel_idx, 4)) return CSA_ERR_ALIGN;
    return from_cuda(csa::launch_attend(*cache, q, n_queries, heads, q_offsets, nullptr, sel_idx, topk, win_kv,
                                        win_start, win_len, max_win, softmax_scale, out, lse, workspace, num_sms(),
                                        reinterpret_cast<cudaStream_t>(stream)));
}

csa_status hca_decode_attend(const csa_cache *cache, const void *q, int32_t n_queries, int32_t heads,
                             const int32_t *q_offsets, const int32_t *q_pos, const void *win_kv,
                             const int64_t *win_start, const int32_t *win_len, int32_t max_win, float softmax_scale,
                             float *out, float *lse, void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    csa_status st = check_attend(cache, q, n_queries, heads, q_offsets, win_kv, win_start, win_len, max_win, out, lse,
                                 workspace, workspace_bytes);
    if (st != CSA_OK) return st;
    if (!q_pos) return CSA_ERR_NULL;
    if (!aligned(q_pos, 4)) return CSA_ERR_ALIGN;
    return from_cuda(csa::launch_attend(*cache, q, n_queries, heads, q_offsets, q_pos, nullptr, 0, win_kv, win_start,
                                        win_len, max_win, softmax_scale, out, lse, workspace, num_sms(),
                                        reinterpret_cast<cudaStream_t>(stream)));
}

csa_status csa_read_device_status(const csa_cache *cache, csa_stream_t stream, int32_t *out_flags) {
    if (!cache || !cache->status || !out_flags) return CSA_ERR_NULL;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return CSA_ERR_CUDA;
    int32_t v = 0, zero = 0;
    if (cudaMemcpy(&v, cache->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return CSA_ERR_CUDA;
    if (cudaMemcpy(cache->status, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return CSA_ERR_CUDA;
    *out_flags = v;
    return CSA_OK;
}

size_t hca_shared_attend_workspace(const csa_cache *cache, int32_t n_queries, int32_t heads) {
    if (!cache || cache->batch < 1 || n_queries < 1 || heads < 1 || heads > 64 ||
        (cache->dim != 128 && cache->dim != 512))
        return 0;
    const int sms = num_sms();
    if (sms <= 0) return 0;
    return csa::shared_attend_workspace_bytes(cache->batch, n_queries, heads, cache->dim, sms);
}

csa_status hca_shared_attend(const csa_cache *cache, const void *q, int32_t n_queries, int32_t heads,
                             const int32_t *q_offsets, const int32_t *q_pos, const float *join_out,
                             const float *join_lse, float softmax_scale, void *out, float *lse, void *workspace,
                             size_t workspace_bytes, csa_stream_t stream) {
    csa_status st = check_cache(cache);
    if (st != CSA_OK) return st;
    if (!q || !q_offsets || !out || (join_out == nullptr) != (join_lse == nullptr)) return CSA_ERR_NULL;
    if (n_queries < 1 || heads < 1) return CSA_ERR_SHAPE;
    if (heads > 64 || (cache->dim != 128 && cache->dim != 512)) return CSA_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(join_out, 16) || !aligned(q_offsets, 4) || !aligned(q_pos, 4) ||
        !aligned(join_lse, 4) || !aligned(lse, 4))
        return CSA_ERR_ALIGN;
    const int64_t vec = (int64_t)n_queries * heads, n2 = 2 * vec * cache->dim, n4 = 2 * n2;
    if (ranges_meet(out, n2, q, n2) || ranges_meet(out, n2, join_out, n4) || ranges_meet(out, n2, join_lse, 4 * vec) ||
        ranges_meet(out, n2, lse, 4 * vec) || ranges_meet(lse, 4 * vec, q, n2) ||
        ranges_meet(lse, 4 * vec, join_out, n4) || ranges_meet(lse, 4 * vec, join_lse, 4 * vec))
        return CSA_ERR_SHAPE;
    const size_t need = hca_shared_attend_workspace(cache, n_queries, heads);
    if (need == 0) return CSA_ERR_CUDA;
    if (!workspace || workspace_bytes < need) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    return from_cuda(csa::launch_shared_attend(*cache, q, n_queries, heads, q_offsets, q_pos, join_out, join_lse,
                                               softmax_scale, out, lse, workspace, num_sms(),
                                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t csa_cache_copy_workspace(const csa_cache *dst, int32_t n_jobs, int32_t keep_cols) {
    if (!dst || dst->batch < 1 || n_jobs < 0 || n_jobs > kMaxCopyJobs || keep_cols < 0 || keep_cols > kMaxCapacity)
        return 0;
    return csa::cache_copy_workspace_bytes(dst->batch, n_jobs, keep_cols);
}

csa_status csa_cache_copy(const csa_cache *src, const csa_cache *dst, int32_t n_jobs, const int32_t *src_slot,
                          const int32_t *dst_slot, const int32_t *keep, int32_t keep_cols, const int32_t *max_blocks,
                          void *workspace, size_t workspace_bytes, csa_stream_t stream) {
    csa_status st = check_cache(src);
    if (st != CSA_OK) return st;
    if ((st = check_cache(dst)) != CSA_OK) return st;
    if (n_jobs < 0 || keep_cols < 0) return CSA_ERR_SHAPE;
    if (n_jobs > 0 && (keep == nullptr) != (keep_cols == 0)) return CSA_ERR_SHAPE;  // (no jobs: a list without an address)
    if (src->dim != dst->dim || src->block != dst->block || src->scale_fmt != dst->scale_fmt ||
        (src->idx_key == nullptr) != (dst->idx_key == nullptr))
        return CSA_ERR_SHAPE;
    if (src->idx_key && (src->idx_dim != dst->idx_dim || src->idx_dtype != dst->idx_dtype)) return CSA_ERR_SHAPE;
    if (n_jobs > kMaxCopyJobs || keep_cols > kMaxCapacity || src->dim > kMaxCopyDim) return CSA_ERR_UNSUPPORTED;
    if (!same_or_apart(*src, *dst)) return CSA_ERR_SHAPE;
    if (n_jobs == 0) return CSA_OK;
    if (!src_slot || !dst_slot) return CSA_ERR_NULL;
    if (!aligned(src_slot, 4) || !aligned(dst_slot, 4) || !aligned(keep, 4) || !aligned(max_blocks, 4))
        return CSA_ERR_ALIGN;
    if (!workspace || workspace_bytes < csa_cache_copy_workspace(dst, n_jobs, keep_cols)) return CSA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return CSA_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return CSA_ERR_CUDA;
    return from_cuda(csa::launch_cache_copy(*src, *dst, n_jobs, src_slot, dst_slot, keep, keep_cols, max_blocks,
                                            workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
}

csa_status csa_rotary(const csa_vectors *x, const csa_vectors *out, int32_t rows, int32_t heads, int32_t dim,
                      const csa_rope *rope, const int32_t *pos, int32_t inverse, csa_stream_t stream) {
    if (!x || !out || !rope) return CSA_ERR_NULL;
    if (rows < 0 || heads < 1 || dim < 2) return CSA_ERR_SHAPE;
    if (rope->rot_begin < 0 || rope->rot_dim < 2 || rope->rot_dim % 2 != 0 || rope->rot_begin > dim - rope->rot_dim)
        return CSA_ERR_SHAPE;
    if (rope->layout != CSA_ROPE_PAIRS && rope->layout != CSA_ROPE_HALF) return CSA_ERR_SHAPE;
    if (!dtype_ok(x->dtype) || !dtype_ok(out->dtype)) return CSA_ERR_SHAPE;
    if (dim > kMaxRotaryDim) return CSA_ERR_UNSUPPORTED;
    if (rows == 0) return CSA_OK;
    if (!x->data || !out->data || !rope->inv_freq || !pos) return CSA_ERR_NULL;
    if (!aligned(x->data, dtype_size(x->dtype)) || !aligned(out->data, dtype_size(out->dtype)) ||
        !aligned(rope->inv_freq, 4) || !aligned(pos, 4))
        return CSA_ERR_ALIGN;
    const VectorShape shape = {rows, heads, dim};
    if (!strides_ok(*x, shape) || !strides_ok(*out, shape) || self_overlap(*out, shape)) return CSA_ERR_SHAPE;
    const bool in_place = x->data == out->data && same_layout(*x, *out, shape);
    if (!in_place && overlap(*x, *out, shape)) return CSA_ERR_SHAPE;
    return from_cuda(csa::launch_rotary(*x, *out, rows, heads, dim, *rope, pos, inverse != 0, in_place,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

csa_status csa_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, int32_t original_len,
                                  double beta_fast, double beta_slow, float *inv_freq, float *mscale) {
    if (!inv_freq) return CSA_ERR_NULL;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > kMaxRotaryDim || !(base > 1.0) || std::isinf(base))
        return CSA_ERR_SHAPE;
    if (scaling < CSA_ROPE_SCALE_NONE || scaling > CSA_ROPE_SCALE_PARTS) return CSA_ERR_SHAPE;
    if (scaling != CSA_ROPE_SCALE_NONE && (!(factor >= 1.0) || std::isinf(factor))) return CSA_ERR_SHAPE;
    if (scaling == CSA_ROPE_SCALE_BASE) {
        if (rot_dim <= 2) return CSA_ERR_SHAPE;
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    }
    double low = 0, high = 0;
    if (scaling == CSA_ROPE_SCALE_PARTS) {
        if (original_len < 1 || !(beta_slow > 0) || !(beta_fast >= beta_slow) || std::isinf(beta_fast))
            return CSA_ERR_SHAPE;
        // the pair that turns `beta` times in original_len tokens: original_len * f_p = 2 pi beta
        auto pair_of = [&](double beta) {
            return rot_dim * std::log(original_len / (2 * 3.14159265358979323846 * beta)) / (2 * std::log(base));
        };
        low = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(beta_slow)), rot_dim - 1.0);
    }
    for (int p = 0; p < rot_dim / 2; ++p) {
        double f = std::pow(base, -2.0 * p / rot_dim);
        if (scaling == CSA_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == CSA_ROPE_SCALE_PARTS) {
            const double ramp = std::fmin(std::fmax((p - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f / factor * ramp + f * (1 - ramp);
        }
        inv_freq[p] = (float)f;
    }
    if (mscale) *mscale = scaling == CSA_ROPE_SCALE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return CSA_OK;
}

csa_status csa_probe_mxf4_mma(int32_t iters, int32_t *status, csa_stream_t stream, int64_t *flops) {
    if (!status || !flops) return CSA_ERR_NULL;
    if (iters < 1) return CSA_ERR_SHAPE;
    if (!aligned(status, 4)) return CSA_ERR_ALIGN;
    const int sms = num_sms();
    if (sms <= 0) return CSA_ERR_CUDA;
    *flops = (int64_t)sms * iters * 2 * 128 * 256 * 128;
    return from_cuda(csa::launch_mxf4_probe(iters, status, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
