// key_weights.cu -- accumulated attention weights (attn_key_weights,
// attn_key_weights_paged): the column sums of the attention matrix.
#include "common.cuh"
#include "kernels.h"
#include "key_weights.h"
#include "plan.h"

using namespace vgqa;

namespace {

int key_weights(attn_plan_t plan, const void *q, long long T_q, const void *k, long long k_stride, long long T_kv, const Paging *pg,
                const int32_t *cu_q, const int32_t *cu_k, const float *lse, float decay, const float *weight_in,
                float *weight_out, int64_t ld, const int32_t *seen, int32_t *born, void *stream) {
    // tensors without rows have no address; none of these is read then
    if (T_q == 0 && !q) q = plan->scratch;
    if (T_q == 0 && !lse) lse = static_cast<const float *>(plan->scratch);
    if (!pg && T_kv == 0 && !k) k = plan->scratch;
    if (!q || !k || !cu_q || !cu_k || !lse || !weight_out || !seen != !born) return ATTN_E_NULL;
    if (!aligned(q, 16) || !aligned(k, 16)) return ATTN_E_ALIGNMENT;
    for (const void *ptr : {(const void *)cu_q, (const void *)cu_k, (const void *)lse, (const void *)weight_in,
                            (const void *)weight_out, (const void *)seen, (const void *)born})
        if (!aligned(ptr, 4)) return ATTN_E_ALIGNMENT;
    const attn_plan_desc &d = plan->d;
    if (T_q < 0 || T_q >= (1ll << 31) || T_kv < 0 || T_kv >= (1ll << 31)) return ATTN_E_INVALID_ARG;
    if (ld < d.s_max || ld > (1ll << 38) || !(decay >= 0.f) || decay > 3.4e38f) return ATTN_E_INVALID_ARG;
    // the sums may take the place of what they add to, but not overlap it
    // otherwise, nor the births
    const size_t led = (size_t)d.B_max * d.Hkv * ld * 4;
    auto overlap = [&](const void *x, const void *y) {
        return x && y && static_cast<const char *>(x) < static_cast<const char *>(y) + led &&
               static_cast<const char *>(y) < static_cast<const char *>(x) + led;
    };
    if ((weight_in != weight_out && overlap(weight_in, weight_out)) || overlap(born, weight_out) ||
        overlap(born, weight_in))
        return ATTN_E_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_E_CUDA;
    if (dev != plan->device) return ATTN_E_DEVICE;

    Params p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.lse = const_cast<float *>(lse);
    p.err = plan->err;
    p.wait_ns = plan->wait_ns;
    p.rows_q = (int)T_q;
    if (!pg) p.rows_kv = (int)T_kv;
    p.B_max = d.B_max;
    p.s_max = d.s_max;
    p.Hq = d.Hq;
    p.Hkv = d.Hkv;
    p.D = d.D;
    p.max_q = d.max_q;
    p.G = d.G;
    p.scale_log2 = plan->scale_log2;
    p.k_stride = k_stride;
    if (pg) {
        p.block_table = pg->block_table;
        p.bt_stride = pg->bt_stride;
        p.page_shift = log2_exact(pg->page_size);
        p.num_pages = pg->num_pages;
        p.page_box = pg->page_size < 64 ? pg->page_size : 64;
        p.page_stride = pg->page_stride;
    }
    KeyWeights kw{weight_in, weight_out, seen, born, ld, decay, plan->kw_part, plan->kw_ticket};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!plan->kw_columns) return launch_key_weights_simt(p, kw, s) == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;

    p.qtile = plan->kw_qtile;
    CUtensorMap tm_q, tm_k;
    // the maps end where the buffers end, and no box starts before their first row
    int rc = encode_q_map(&tm_q, q, d.Hq, d.D, d.G, p.qtile, T_q > 0 ? T_q : 1);
    if (rc != ATTN_OK) return rc;
    if (pg) {
        // pages a whole number of token rows apart: one row index per key
        if (pg->page_stride % k_stride == 0 && (long long)pg->num_pages * (pg->page_stride / k_stride) < (1ll << 31))
            p.page_rows = (int)(pg->page_stride / k_stride);
        rc = p.page_rows ? encode_kv_map(&tm_k, k, d.Hkv, d.D, p.page_box, k_stride,
                                         (long long)pg->num_pages * p.page_rows)
                         : encode_paged_map(&tm_k, k, d.Hkv, d.D, pg->page_size, pg->num_pages, k_stride,
                                            pg->page_stride);
    } else {
        rc = encode_kv_map(&tm_k, k, d.Hkv, d.D, 128, k_stride, T_kv > 0 ? T_kv : 1);
    }
    if (rc != ATTN_OK) return rc;
    const cudaError_t e = launch_key_weights_tc(p, kw, tm_q, tm_k, plan->kw_columns, plan->kw_ctas, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;
}

}  // namespace

ATTN_EXPORT int attn_key_weights(attn_plan_t plan, const void *q, int64_t T_q, const void *k, int64_t k_token_stride,
                                 int64_t T_kv, const int32_t *cu_q, const int32_t *cu_k, const float *lse, float decay,
                                 const float *weight_in, float *weight_out, int64_t ld, const int32_t *seen,
                                 int32_t *born, void *stream) {
    if (!plan || !live(plan)) return ATTN_E_BAD_PLAN;
    const long long packed = (long long)plan->d.Hkv * plan->d.D;
    if (k_token_stride < packed || k_token_stride % 8 != 0 || k_token_stride > (1ll << 38)) return ATTN_E_INVALID_ARG;
    return key_weights(plan, q, T_q, k, k_token_stride, T_kv, nullptr, cu_q, cu_k, lse, decay, weight_in, weight_out, ld, seen,
                       born, stream);
}

ATTN_EXPORT int attn_key_weights_paged(attn_plan_t plan, const void *q, int64_t T_q, const void *k_cache, int64_t page_stride,
                                       int64_t token_stride, int page_size, int num_pages, const int32_t *block_table,
                                       int bt_stride, const int32_t *cu_q, const int32_t *cu_k, const float *lse,
                                       float decay, const float *weight_in, float *weight_out, int64_t ld,
                                       const int32_t *seen, int32_t *born, void *stream) {
    if (!plan || !live(plan)) return ATTN_E_BAD_PLAN;
    const int rc = check_paging(plan, page_stride, token_stride, page_size, num_pages, block_table, bt_stride);
    if (rc != ATTN_OK) return rc;
    const Paging pg{block_table, bt_stride, page_size, num_pages, page_stride};
    return key_weights(plan, q, T_q, k_cache, token_stride, 0, &pg, cu_q, cu_k, lse, decay, weight_in, weight_out, ld, seen,
                       born, stream);
}
