// api_cache.cu -- the C ABI of the calls on new tokens (norm and rotation,
// append, chunk attention) and on e4m3 caches (declared in
// include/longspec_hta.h).  Host side only: argument checks and launches.
#include <cmath>

#include "../../include/longspec_hta.h"
#include "api_internal.h"
#include "cache_kernels.h"
#include "hta_kernels.h"

using namespace hta_api;

namespace {

constexpr long long kIntLimit = 1LL << 31;

// Sizes of a call on N = dims->T ragged tokens (no tree-size limit).
int check_token_dims(const longspec_hta_dims *d) {
    if (!d) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->T < 0 || d->L_cap < 0 || d->Hq % d->Hkv != 0)
        return LONGSPEC_HTA_ERR_INVALID_DIMS;
    if (!(d->scale >= 0.f) || std::isinf(d->scale)) return LONGSPEC_HTA_ERR_INVALID_DIMS;
    if (d->D != 64 && d->D != 128) return LONGSPEC_HTA_ERR_UNSUPPORTED_D;
    if (1LL * d->T * d->Hq >= kIntLimit || 1LL * d->B * d->Hkv > 65535) return LONGSPEC_HTA_ERR_INVALID_DIMS;
    return LONGSPEC_HTA_OK;
}

int check_cache(const longspec_hta_cache *c, const longspec_hta_dims *d) {
    if (!c || !c->k_cache || !c->v_cache || !c->block_table) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned16(c->k_cache) || !aligned16(c->v_cache) || !aligned4(c->block_table))
        return LONGSPEC_HTA_ERR_MISALIGNED;
    if ((c->k_scale == nullptr) != (c->v_scale == nullptr)) return LONGSPEC_HTA_ERR_INVALID_OPTION;
    if (!aligned16(c->k_scale) || !aligned16(c->v_scale)) return LONGSPEC_HTA_ERR_MISALIGNED;
    const int bs = c->block_size;
    if ((bs != 16 && bs != 32 && bs != 64 && bs != 128) || c->num_blocks < 1 || c->max_blocks < 1 ||
        1LL * c->max_blocks * bs < d->L_cap || 1LL * c->max_blocks * bs >= kIntLimit ||
        1LL * c->num_blocks * d->Hkv * bs + 128 >= kIntLimit)
        return LONGSPEC_HTA_ERR_INVALID_DIMS;
    return LONGSPEC_HTA_OK;
}

int check_heads(const longspec_hta_heads *h) {
    if (!h || !h->p) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned16(h->p) || ((h->stride_b | h->stride_t | h->stride_h) & 7) != 0) return LONGSPEC_HTA_ERR_MISALIGNED;
    return LONGSPEC_HTA_OK;
}

int check_rope(const longspec_hta_rope *r, int D) {
    if (!r || !r->inv_freq) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned4(r->inv_freq) || !aligned16(r->q_weight) || !aligned16(r->k_weight))
        return LONGSPEC_HTA_ERR_MISALIGNED;
    if (r->rot_dim < 2 || r->rot_dim > D || r->rot_dim % 2 != 0 || !(r->scale >= 0.f) || std::isinf(r->scale) ||
        !(r->eps >= 0.f) || std::isinf(r->eps))
        return LONGSPEC_HTA_ERR_INVALID_OPTION;
    return LONGSPEC_HTA_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (!ws) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned16(ws)) return LONGSPEC_HTA_ERR_MISALIGNED;
    return bytes < need ? LONGSPEC_HTA_ERR_WORKSPACE_TOO_SMALL : LONGSPEC_HTA_OK;
}

int check_ints(const void *p) {
    return !p ? LONGSPEC_HTA_ERR_NULL_POINTER : aligned4(p) ? LONGSPEC_HTA_OK : LONGSPEC_HTA_ERR_MISALIGNED;
}

#define HTA_TRY(x) do { const int rc_ = (x); if (rc_) return rc_; } while (0)

hta::HeadRows rows_of(const longspec_hta_heads *h) {
    return {static_cast<__nv_bfloat16 *>(h->p), h->stride_b, h->stride_h, h->stride_t};
}

hta::CacheView view_of(const longspec_hta_cache *c) {
    return {c->k_cache, c->v_cache, c->k_scale, c->v_scale, c->block_table, c->block_size, c->max_blocks,
            c->num_blocks};
}

void set_rope(hta::RowsParams *p, const longspec_hta_rope *r) {
    p->rotate = 1;
    p->rot_dim = r->rot_dim;
    p->interleaved = r->interleaved != 0;
    p->inv_freq = r->inv_freq;
    p->rope_scale = r->scale > 0.f ? r->scale : 1.f;
    p->eps = r->eps;
    p->q_weight = static_cast<const __nv_bfloat16 *>(r->q_weight);
    p->k_weight = static_cast<const __nv_bfloat16 *>(r->k_weight);
}

// Workspace of the attention calls: status word, partial headers, and two
// slots of up to 256 rows per CTA (chunk_tc.cu).
struct SlotLayout {
    int slot_rows;
    size_t heads_off, o_off, lse_off, total;
};
SlotLayout slot_layout(long long packed_rows, int D, int grid) {
    SlotLayout l;
    l.slot_rows = static_cast<int>(packed_rows < 256 ? packed_rows : 256);
    l.heads_off = hta::kStatusBytes;
    l.o_off = align256(l.heads_off + 2 * sizeof(hta::PartHead) * grid);
    l.lse_off = align256(l.o_off + 2ull * grid * l.slot_rows * D * sizeof(float));
    l.total = align256(l.lse_off + 2ull * grid * l.slot_rows * sizeof(float));
    return l;
}

// Rows [rows][D] of bf16 in boxes of 64 columns, 128-byte swizzle, or of e4m3
// codes in whole rows.
int rows_map(const void *base, uint64_t rows, int D, int box_rows, bool q8, CUtensorMap *out,
             CUtensorMapSwizzle q8_swizzle = CU_TENSOR_MAP_SWIZZLE_NONE) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return LONGSPEC_HTA_ERR_CUDA;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), rows};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * (q8 ? 1 : 2)};
    const cuuint32_t box[2] = {q8 ? static_cast<cuuint32_t>(D) : 64u, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
    return fn(out, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base),
              dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              q8 ? q8_swizzle : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LONGSPEC_HTA_OK : LONGSPEC_HTA_ERR_CUDA;
}

// The common part of the attention calls: p holds the rows, the lengths and
// the outputs already.
int run_attention(hta::ChunkParams &p, const longspec_hta_dims *d, const longspec_hta_cache *cache, void *workspace,
                  int num_sms, cudaStream_t stream) {
    p.B = d->B; p.Hq = d->Hq; p.Hkv = d->Hkv; p.G = d->Hq / d->Hkv; p.D = d->D;
    p.N = d->T;
    p.L_cap = d->L_cap;
    p.scale_log2 = scale_of(d) * hta::kLog2e;
    p.cache = view_of(cache);
    p.grid = num_sms;
    const SlotLayout l = slot_layout(1LL * p.G * d->T, d->D, p.grid);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.slot_rows = l.slot_rows;
    p.status = reinterpret_cast<uint32_t *>(ws);
    p.heads = reinterpret_cast<hta::PartHead *>(ws + l.heads_off);
    p.o_part = reinterpret_cast<float *>(ws + l.o_off);
    p.lse_part = reinterpret_cast<float *>(ws + l.lse_off);
    CUtensorMap tm[4] = {};
    const uint64_t cache_rows = 1ull * cache->num_blocks * d->Hkv * cache->block_size;
    const bool q8 = cache->k_scale != nullptr;
    p.g_shift = 0;
    while ((1 << p.g_shift) < p.G) ++p.g_shift;
    p.g_mul = static_cast<uint32_t>((1ull << (31 + p.g_shift)) / p.G + 1);
    // The kernel for few rows of a sequence, over an e4m3 cache.  It reads the keys
    // once for every 8 rows (16 where chunk_decode.cu says so), against once for up to
    // 128 or 256, and the host knows the rows on average only:
    //   a token a sequence, up to 16 heads a KV head: 32 x 8k keys, 8 heads 60 us
    //     against 112, 16 heads 108 against 113, one sequence of 128k 60 against 70;
    //   up to 8 rows on average: 64 x 2 tokens of 4 heads over 4k keys 114 against
    //     221, 63 tokens and a chunk of 40 143 against 239 (but 63 tokens of 100 keys
    //     and a chunk of 65 at 64k 1656 against 209);
    //   more rows gain little (12 rows: D = 128 107 against 113, D = 64 67 against 94),
    //     and a long chunk among single tokens loses by as much as it is long (63
    //     tokens and a chunk of 193, 4k keys: 762 against 260).  So does one chunk among
    //     empty sequences, which T and B do not tell from single tokens.
    const bool few = q8 && !p.tree && (d->T <= d->B ? p.G <= 16 : 1LL * d->T * p.G <= 8LL * d->B);
    const CUtensorMapSwizzle sw = !few ? CU_TENSOR_MAP_SWIZZLE_NONE
                                  : d->D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    HTA_TRY(rows_map(cache->k_cache, cache_rows, d->D, cache->block_size, q8, &tm[0], sw));
    HTA_TRY(rows_map(cache->v_cache, cache_rows, d->D, cache->block_size, q8, &tm[1], sw));
    if (few) return hta::launch_chunk_decode(p, tm, stream) == cudaSuccess ? LONGSPEC_HTA_OK : LONGSPEC_HTA_ERR_CUDA;
    if (p.tree_tiles) {
        const uint64_t rows = 1ull * d->B * d->Hkv * d->T;
        HTA_TRY(rows_map(p.k_tree, rows, d->D, 128, false, &tm[2]));
        HTA_TRY(rows_map(p.v_tree, rows, d->D, 128, false, &tm[3]));
    }
    return hta::launch_chunk_tc(p, tm, stream) == cudaSuccess ? LONGSPEC_HTA_OK : LONGSPEC_HTA_ERR_CUDA;
}

int done(cudaError_t e) { return e == cudaSuccess ? LONGSPEC_HTA_OK : LONGSPEC_HTA_ERR_CUDA; }

}  // namespace

extern "C" {

int longspec_hta_qk_norm_rope(int B, int T, int Hq, int Hkv, int D, const longspec_hta_heads *q,
                              const longspec_hta_heads *k, const int32_t *positions, const longspec_hta_rope *rope,
                              const longspec_hta_heads *q_out, const longspec_hta_heads *k_out,
                              cudaStream_t stream) {
    if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || 1LL * B * T >= kIntLimit ||
        1LL * B * T * (Hq > Hkv ? Hq : Hkv) >= kIntLimit)
        return LONGSPEC_HTA_ERR_INVALID_DIMS;
    if (D != 64 && D != 128) return LONGSPEC_HTA_ERR_UNSUPPORTED_D;
    HTA_TRY(check_rope(rope, D));
    if (B == 0 || T == 0) return LONGSPEC_HTA_OK;
    HTA_TRY(check_heads(q));
    HTA_TRY(check_heads(k));
    HTA_TRY(check_heads(q_out));
    HTA_TRY(check_heads(k_out));
    HTA_TRY(check_ints(positions));
    DeviceInfo di;
    HTA_TRY(current_device(&di));
    hta::RowsParams p{};
    p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.T = T;
    p.tokens = B * T;
    p.q = rows_of(q); p.k = rows_of(k);
    p.q_out = rows_of(q_out); p.k_out = rows_of(k_out);
    p.positions = positions;
    set_rope(&p, rope);
    return done(hta::launch_rows(p, di.num_sms, stream));
}

int longspec_hta_append_paged(const longspec_hta_dims *dims, const longspec_hta_heads *q, const longspec_hta_heads *k,
                              const longspec_hta_heads *v, const longspec_hta_rope *rope,
                              const longspec_hta_cache *cache, const int32_t *prefix_len, const int32_t *q_start,
                              const longspec_hta_heads *q_out, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    HTA_TRY(check_token_dims(dims));
    HTA_TRY(check_cache(cache, dims));
    if (rope) HTA_TRY(check_rope(rope, dims->D));
    HTA_TRY(check_ints(prefix_len));
    HTA_TRY(check_ints(q_start));
    HTA_TRY(check_workspace(workspace, workspace_bytes, hta::kStatusBytes));
    if (dims->T == 0) return LONGSPEC_HTA_OK;
    HTA_TRY(check_heads(k));
    HTA_TRY(check_heads(v));
    if (rope) {
        HTA_TRY(check_heads(q));
        HTA_TRY(check_heads(q_out));
    }
    DeviceInfo di;
    HTA_TRY(current_device(&di));
    hta::RowsParams p{};
    p.Hq = dims->Hq; p.Hkv = dims->Hkv; p.D = dims->D; p.T = dims->T;
    p.tokens = dims->T;
    p.k = rows_of(k); p.v = rows_of(v);
    if (rope) {
        p.q = rows_of(q);
        p.q_out = rows_of(q_out);
        set_rope(&p, rope);
    }
    p.cache = view_of(cache);
    p.prefix_len = prefix_len;
    p.q_start = q_start;
    p.B = dims->B;
    p.L_cap = dims->L_cap;
    p.status = static_cast<uint32_t *>(workspace);
    return done(hta::launch_rows(p, di.num_sms, stream));
}

size_t longspec_hta_chunk_workspace_bytes(const longspec_hta_dims *dims) {
    DeviceInfo di;
    if (check_token_dims(dims) != LONGSPEC_HTA_OK || current_device(&di) != LONGSPEC_HTA_OK) return 0;
    return slot_layout(1LL * (dims->Hq / dims->Hkv) * dims->T, dims->D, di.num_sms).total;
}

int longspec_hta_chunk_attention_paged(const longspec_hta_dims *dims, const longspec_hta_heads *q,
                                       const longspec_hta_cache *cache, const int32_t *prefix_len,
                                       const int32_t *q_start, int window, void *out, float *lse, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
    HTA_TRY(check_token_dims(dims));
    HTA_TRY(check_cache(cache, dims));
    HTA_TRY(check_ints(prefix_len));
    HTA_TRY(check_ints(q_start));
    if (window < 0) return LONGSPEC_HTA_ERR_INVALID_OPTION;
    HTA_TRY(check_workspace(workspace, workspace_bytes, hta::kStatusBytes));
    if (dims->T == 0) return LONGSPEC_HTA_OK;
    HTA_TRY(check_heads(q));
    if (dims->Hq > 1 && q->stride_h != dims->D) return LONGSPEC_HTA_ERR_INVALID_OPTION;
    if (!out || !lse) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned16(out) || !aligned4(lse)) return LONGSPEC_HTA_ERR_MISALIGNED;
    DeviceInfo di;
    HTA_TRY(current_device(&di));
    HTA_TRY(check_workspace(workspace, workspace_bytes, longspec_hta_chunk_workspace_bytes(dims)));
    hta::ChunkParams p{};
    p.window = window;
    p.q = static_cast<const __nv_bfloat16 *>(q->p);
    p.q_stride = q->stride_t;
    p.prefix_len = prefix_len;
    p.q_start = q_start;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    return run_attention(p, dims, cache, workspace, di.num_sms, stream);
}

size_t longspec_hta_q8_workspace_bytes(const longspec_hta_dims *dims) {
    DeviceInfo di;
    if (check_dims(dims) != LONGSPEC_HTA_OK || current_device(&di) != LONGSPEC_HTA_OK) return 0;
    return slot_layout(1LL * (dims->Hq / dims->Hkv) * dims->T, dims->D, di.num_sms).total;
}

static int run_q8(const longspec_hta_dims *dims, const void *q, const longspec_hta_cache *cache,
                  const int32_t *prefix_len, const void *k_tree, const void *v_tree, const int32_t *parent, void *out,
                  float *lse, void *workspace, size_t workspace_bytes, bool prefix_only, cudaStream_t stream) {
    HTA_TRY(check_dims(dims));
    HTA_TRY(check_cache(cache, dims));
    if (!cache->k_scale) return LONGSPEC_HTA_ERR_INVALID_OPTION;
    const void *ptrs[] = {q, prefix_len, out, lse, prefix_only ? q : k_tree, prefix_only ? q : v_tree,
                          prefix_only ? q : parent};
    for (const void *x : ptrs) {
        if (!x) return LONGSPEC_HTA_ERR_NULL_POINTER;
        if (!aligned16(x)) return LONGSPEC_HTA_ERR_MISALIGNED;
    }
    HTA_TRY(check_workspace(workspace, workspace_bytes, hta::kStatusBytes));
    DeviceInfo di;
    HTA_TRY(current_device(&di));
    HTA_TRY(check_workspace(workspace, workspace_bytes, longspec_hta_q8_workspace_bytes(dims)));
    hta::ChunkParams p{};
    p.tree = 1;
    p.tree_tiles = prefix_only ? 0 : (dims->T + 127) / 128;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.prefix_len = prefix_len;
    p.k_tree = static_cast<const __nv_bfloat16 *>(k_tree);
    p.v_tree = static_cast<const __nv_bfloat16 *>(v_tree);
    p.parent = parent;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    return run_attention(p, dims, cache, workspace, di.num_sms, stream);
}

int longspec_hta_verify_paged_q8(const longspec_hta_dims *dims, const void *q, const longspec_hta_cache *cache,
                                 const int32_t *prefix_len, const void *k_tree, const void *v_tree,
                                 const int32_t *parent, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    return run_q8(dims, q, cache, prefix_len, k_tree, v_tree, parent, out, lse, workspace, workspace_bytes, false,
                  stream);
}

int longspec_hta_prefix_attention_paged_q8(const longspec_hta_dims *dims, const void *q,
                                           const longspec_hta_cache *cache, const int32_t *prefix_len, void *out,
                                           float *lse, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return run_q8(dims, q, cache, prefix_len, nullptr, nullptr, nullptr, out, lse, workspace, workspace_bytes, true,
                  stream);
}

int longspec_hta_commit_paged_q8(const longspec_hta_dims *dims, const longspec_hta_cache *cache, int32_t *prefix_len,
                                 const void *k_tree, const void *v_tree, const int32_t *accept_len,
                                 const int32_t *path, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    HTA_TRY(check_dims(dims));
    HTA_TRY(check_cache(cache, dims));
    if (!cache->k_scale) return LONGSPEC_HTA_ERR_INVALID_OPTION;
    if (!k_tree || !v_tree) return LONGSPEC_HTA_ERR_NULL_POINTER;
    if (!aligned16(k_tree) || !aligned16(v_tree)) return LONGSPEC_HTA_ERR_MISALIGNED;
    HTA_TRY(check_ints(prefix_len));
    HTA_TRY(check_ints(accept_len));
    HTA_TRY(check_ints(path));
    HTA_TRY(check_workspace(workspace, workspace_bytes, hta::kStatusBytes));
    DeviceInfo di;
    HTA_TRY(current_device(&di));
    hta::CommitQ8Params p{};
    p.B = dims->B; p.Hkv = dims->Hkv; p.D = dims->D; p.T = dims->T; p.L_cap = dims->L_cap;
    p.cache = view_of(cache);
    p.prefix_len = prefix_len;
    p.k_tree = static_cast<const __nv_bfloat16 *>(k_tree);
    p.v_tree = static_cast<const __nv_bfloat16 *>(v_tree);
    p.accept_len = accept_len;
    p.path = path;
    p.status = static_cast<uint32_t *>(workspace);
    return done(hta::launch_commit_q8(p, stream));
}

}  // extern "C"
