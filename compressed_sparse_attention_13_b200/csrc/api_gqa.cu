// C-ABI entry points of the grouped-head attention (declared in
// include/csa.h): argument checks on the host, workspace layout, and the
// choice of kernel for each format.
#include "api_common.h"
#include "kernels.h"

namespace csa {

constexpr uint32_t kGqaFlags = CSA_FLAG_BATCH_INVARIANT | CSA_FLAG_ROT_PAIRS;

static int check_gqa(const csa_gqa_params* p, bool paged) {
    if (!p) return CSA_ERR_ARG;
    if (p->n_heads <= 0 || p->n_kv_heads <= 0 || p->n_heads % p->n_kv_heads) return CSA_ERR_ARG;
    if (p->head_dim <= 0 || p->head_dim % 64 || p->window < 0) return CSA_ERR_ARG;
    if (!act_ok(p->act_fmt) || !(p->scale == p->scale) || (p->flags & ~kGqaFlags)) return CSA_ERR_ARG;
    if (paged && (p->page_size <= 0 || !kv_ok(p->cache_fmt))) return CSA_ERR_ARG;
    if (p->head_dim > 256 || p->n_heads / p->n_kv_heads > 128 || p->n_heads > 65535) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static int64_t act_bytes(const csa_gqa_params* p) { return p->act_fmt == CSA_F32 ? 4 : 2; }

// A token stride: room for the heads, and rows that start on 16 bytes.
static int check_ld(const csa_gqa_params* p, int heads, int64_t ld) {
    if (ld < int64_t(heads) * p->head_dim || ld > (int64_t(1) << 36)) return CSA_ERR_ARG;
    return ld * act_bytes(p) % 16 ? CSA_ERR_ALIGN : CSA_OK;
}

static int check_cache(const csa_gqa_params* p, const void* k, const float* ks, const void* v, const float* vs,
                       int64_t n_pages, const int32_t* table, int64_t max_pages) {
    if (n_pages < 0 || max_pages < 0) return CSA_ERR_ARG;
    if (n_pages > INT32_MAX || max_pages > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    if ((n_pages > 0 && (!k || !v)) || (max_pages > 0 && !table)) return CSA_ERR_ARG;
    if (p->cache_fmt == CSA_FP8_S64 && n_pages > 0 && (!ks || !vs)) return CSA_ERR_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(ks) || !aligned16(vs)) return CSA_ERR_ALIGN;
    return CSA_OK;
}

}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_gqa_workspace_size(const csa_gqa_params* p, int32_t op, int32_t n_seq, int64_t n_tokens, int64_t n_ctx) {
    if (op != CSA_OP_PAGED_DECODE && op != CSA_OP_PROMPT_ATTN) return 0;
    if (check_gqa(p, op == CSA_OP_PAGED_DECODE) || n_seq < 0 || n_tokens < 0 || n_ctx < 0) return 0;
    if (op == CSA_OP_PROMPT_ATTN) return 256;
    return (paged_decode_tc_supported(p->act_fmt, p->cache_fmt) ? paged_decode_workspace : paged_decode_simt_workspace)(
        p->n_heads, p->n_kv_heads, p->head_dim, n_seq, n_ctx, (p->flags & CSA_FLAG_BATCH_INVARIANT) != 0);
}

int paged_append(const csa_gqa_params* p, int32_t n_seq, int64_t n_tokens, const int32_t* cu_q,
                 const int64_t* pos0, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                 const void* v, int64_t v_ld, const double* inv_freq, void* q_out, void* k_out,
                 void* k_cache, float* k_scales, void* v_cache, float* v_scales, int64_t n_pages,
                 const int32_t* block_table, int64_t max_pages, csa_stream_t stream) {
    int st = check_gqa(p, true);
    if (st) return st;
    if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 2) return CSA_ERR_ARG;
    if (p->rot_dim % 16) return CSA_ERR_UNSUPPORTED;
    if (n_seq < 0 || n_tokens < 0) return CSA_ERR_ARG;
    if (n_tokens > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    if (!cu_q && n_tokens != n_seq) return CSA_ERR_ARG;
    if (n_seq == 0 || n_tokens == 0) return CSA_OK;
    if (!pos0 || !k || !v || (q && !q_out) || (p->rot_dim > 0 && !inv_freq)) return CSA_ERR_ARG;
    if (q && (st = check_ld(p, p->n_heads, q_ld))) return st;
    if ((st = check_ld(p, p->n_kv_heads, k_ld)) || (st = check_ld(p, p->n_kv_heads, v_ld))) return st;
    // in place: only where a token's rows are where the dense output puts them
    if (q && q_out == q && q_ld != int64_t(p->n_heads) * p->head_dim) return CSA_ERR_ARG;
    if (k_out == k && k_ld != int64_t(p->n_kv_heads) * p->head_dim) return CSA_ERR_ARG;
    if ((st = check_cache(p, k_cache, k_scales, v_cache, v_scales, n_pages, block_table, max_pages))) return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out))
        return CSA_ERR_ALIGN;
    PagedAppendArgs a;
    a.H = p->n_heads; a.HK = p->n_kv_heads; a.D = p->head_dim; a.page_size = p->page_size;
    a.rot_dim = p->rot_dim; a.rot_pairs = (p->flags & CSA_FLAG_ROT_PAIRS) != 0;
    a.act_fmt = p->act_fmt; a.cache_fmt = p->cache_fmt; a.n_seq = n_seq; a.n_tokens = n_tokens;
    a.cu_q = cu_q; a.pos0 = pos0; a.q = q; a.k = k; a.v = v; a.q_ld = q_ld; a.k_ld = k_ld; a.v_ld = v_ld;
    a.inv_freq = inv_freq; a.q_out = q_out; a.k_out = k_out; a.k_cache = k_cache; a.v_cache = v_cache;
    a.k_scales = k_scales; a.v_scales = v_scales; a.n_pages = n_pages; a.max_pages = max_pages;
    a.block_table = block_table;
    return cuda_status(launch_paged_append(a, (cudaStream_t)stream));
}

int paged_decode_attn(const csa_gqa_params* p, int32_t batch, const void* q, int64_t q_ld,
                      const void* k_cache, const float* k_scales, const void* v_cache,
                      const float* v_scales, int64_t n_pages, const int32_t* block_table,
                      int64_t max_pages, const int64_t* q_pos, const float* sinks, void* out,
                      void* workspace, size_t ws_bytes, csa_stream_t stream) {
    int st = check_gqa(p, true);
    if (st) return st;
    if (batch < 0) return CSA_ERR_ARG;
    if (batch == 0) return CSA_OK;
    if (!q || !q_pos || !out) return CSA_ERR_ARG;
    if ((st = check_ld(p, p->n_heads, q_ld))) return st;
    if ((st = check_cache(p, k_cache, k_scales, v_cache, v_scales, n_pages, block_table, max_pages))) return st;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return CSA_ERR_ALIGN;
    // cache rows, and the places of a sequence, are counted in 32 bits
    if (int64_t(batch) * p->n_heads > INT32_MAX || max_pages * p->page_size > INT32_MAX ||
        n_pages * p->n_kv_heads >= (int64_t(1) << 32) / p->page_size)
        return CSA_ERR_UNSUPPORTED;
    if (ws_bytes < csa_gqa_workspace_size(p, CSA_OP_PAGED_DECODE, batch, batch, max_pages * p->page_size))
        return CSA_ERR_WORKSPACE;
    if (!workspace) return CSA_ERR_ARG;
    PagedDecodeArgs a;
    a.H = p->n_heads; a.HK = p->n_kv_heads; a.D = p->head_dim; a.page_size = p->page_size; a.W = p->window;
    a.act_fmt = p->act_fmt; a.cache_fmt = p->cache_fmt; a.invariant = (p->flags & CSA_FLAG_BATCH_INVARIANT) != 0;
    a.scale = p->scale; a.batch = batch; a.q = q; a.q_ld = q_ld; a.k_cache = k_cache; a.v_cache = v_cache;
    a.k_scales = k_scales; a.v_scales = v_scales; a.n_pages = n_pages; a.max_pages = max_pages;
    a.block_table = block_table; a.q_pos = q_pos; a.sinks = sinks; a.out = out;
    return cuda_status(paged_decode_tc_supported(p->act_fmt, p->cache_fmt)
                           ? launch_paged_decode_tc(a, workspace, (cudaStream_t)stream)
                           : launch_paged_decode_simt(a, workspace, (cudaStream_t)stream));
}

int prompt_attn(const csa_gqa_params* p, int32_t n_seq, const void* q, int64_t q_ld, int64_t n_q,
                const void* k, int64_t k_ld, const void* v, int64_t v_ld, int64_t n_k,
                const int32_t* cu_q, const int32_t* cu_k, const float* sinks, void* out,
                void* workspace, size_t ws_bytes, csa_stream_t stream) {
    int st = check_gqa(p, false);
    if (st) return st;
    if (n_seq < 0 || n_q < 0 || n_k < 0) return CSA_ERR_ARG;
    if (n_q > INT32_MAX || n_k > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    if (n_seq == 0 || n_q == 0) return CSA_OK;
    if (!q || (n_k > 0 && (!k || !v)) || !cu_q || !cu_k || !out) return CSA_ERR_ARG;
    if ((st = check_ld(p, p->n_heads, q_ld)) || (st = check_ld(p, p->n_kv_heads, k_ld)) ||
        (st = check_ld(p, p->n_kv_heads, v_ld)))
        return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace))
        return CSA_ERR_ALIGN;
    if (n_q * p->n_heads > INT32_MAX) return CSA_ERR_UNSUPPORTED;
    if (ws_bytes < csa_gqa_workspace_size(p, CSA_OP_PROMPT_ATTN, n_seq, n_q, 0)) return CSA_ERR_WORKSPACE;
    if (!workspace) return CSA_ERR_ARG;
    PromptArgs a;
    a.H = p->n_heads; a.HK = p->n_kv_heads; a.D = p->head_dim; a.W = p->window; a.act_fmt = p->act_fmt;
    a.n_seq = n_seq; a.scale = p->scale; a.q = q; a.k = k; a.v = v; a.q_ld = q_ld; a.k_ld = k_ld; a.v_ld = v_ld;
    a.n_q = n_q; a.n_k = n_k; a.cu_q = cu_q; a.cu_k = cu_k; a.sinks = sinks; a.out = out;
    return cuda_status(prompt_tc_supported(a) ? launch_prompt_tc(a, (cudaStream_t)stream)
                                              : launch_prompt_simt(a, (cudaStream_t)stream));
}

}  // extern "C"
