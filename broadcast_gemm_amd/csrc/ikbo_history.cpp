// ikbo_history.cpp -- the C ABI of the cached user histories declared in include/ikbo.h:
// argument checks, then one or a few launches on the caller's stream with the caller's buffers.
#include "ikbo.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <limits>

#include "hist_internal.h"

using namespace ikbo;

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned4(const void *p) { return aligned(p, 4); }
bool whole_rows(int64_t stride, int dtype) { return stride % (dtype == IKBO_DTYPE_F32 ? 4 : 8) == 0; }
constexpr int64_t kInt = std::numeric_limits<int32_t>::max();
constexpr int kMaxHeads = 4096;

int check_rows(const ikbo_kv4_rows_args *a) {
    if (a == nullptr || a->T < 0 || a->H_kv < 1 || a->num_pages < 1) return IKBO_ERR_INVALID_ARG;
    if (a->dtype != IKBO_DTYPE_BF16 && a->dtype != IKBO_DTYPE_F32) return IKBO_ERR_INVALID_ARG;
    if ((a->head_dim != 64 && a->head_dim != 128) || a->H_kv > kMaxHeads || (int64_t)a->num_pages * IKBO_KV4_PAGE > kInt)
        return IKBO_ERR_UNSUPPORTED;
    if (a->T == 0) return IKBO_OK;
    if (!a->slots || !a->tiles || !a->status) return IKBO_ERR_INVALID_ARG;
    if (!aligned4(a->slots) || !aligned4(a->status) || !aligned(a->tiles, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) ||
        !whole_rows(a->k_token, a->dtype) || !whole_rows(a->k_head, a->dtype) || !whole_rows(a->v_token, a->dtype) ||
        !whole_rows(a->v_head, a->dtype))
        return IKBO_ERR_ALIGNMENT;
    return IKBO_OK;
}

}  // namespace

extern "C" {

int ikbo_kv_status(uint32_t *status, void *stream) {
    if (status == nullptr) return IKBO_ERR_INVALID_ARG;
    hipError_t e = hipStreamSynchronize(static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    uint32_t word = 0;
    if ((e = hipMemcpy(&word, status, sizeof word, hipMemcpyDeviceToHost)) != hipSuccess)
        return hip_fail(e, "hipMemcpy(status)");
    if (word == 0) return IKBO_OK;
    // On the caller's stream, so that what it enqueues next comes behind.
    if ((e = hipMemsetAsync(status, 0, sizeof word, static_cast<hipStream_t>(stream))) != hipSuccess ||
        (e = hipStreamSynchronize(static_cast<hipStream_t>(stream))) != hipSuccess)
        return hip_fail(e, "hipMemset(status)");
    if (word & kStMap) return IKBO_ERR_MAP_RANGE;
    if (word & kStPage) return IKBO_ERR_PAGE_RANGE;
    if (word & kStNoPages) return IKBO_ERR_NO_PAGES;
    return IKBO_ERR_NONFINITE;
}

int ikbo_kv_tables(const ikbo_kv_tables_args *a, void *stream) {
    if (a == nullptr || a->B_u < 1 || a->max_pages < 1 || a->num_pages < 1 || a->page_size < 1 || a->capacity < 0 ||
        a->table_stride < a->max_pages)
        return IKBO_ERR_INVALID_ARG;
    if (a->B_u > IKBO_KV_MAX_USERS || (int64_t)a->num_pages * a->page_size > kInt || (int64_t)a->max_pages * a->page_size > kInt)
        return IKBO_ERR_UNSUPPORTED;
    const void *need[] = {a->counts, a->lens, a->lens_out, a->block_table, a->ring, a->state, a->state_out, a->starts, a->status};
    for (const void *p : need) {
        if (p == nullptr) return IKBO_ERR_INVALID_ARG;
        if (!aligned4(p)) return IKBO_ERR_ALIGNMENT;
    }
    const void *rows[] = {a->slots, a->positions, a->rows};
    for (const void *p : rows) {
        if (p == nullptr && a->capacity > 0) return IKBO_ERR_INVALID_ARG;
        if (!aligned4(p)) return IKBO_ERR_ALIGNMENT;
    }
    const hipError_t e = launch_kv_tables(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "kv tables");
}

int ikbo_rope(const ikbo_rope_args *a, void *stream) {
    if (a == nullptr || a->T < 0 || a->H_q < 0 || a->H_k < 0 || a->H_q + (int64_t)a->H_k < 1 || a->head_dim < 2 || a->rot_dim < 2 ||
        a->rot_dim % 2 != 0 || a->rot_dim > a->head_dim)
        return IKBO_ERR_INVALID_ARG;
    if ((a->layout != IKBO_ROPE_HALF && a->layout != IKBO_ROPE_INTERLEAVED) || (a->inverse != 0 && a->inverse != 1) ||
        (a->dtype != IKBO_DTYPE_BF16 && a->dtype != IKBO_DTYPE_F32) || !std::isfinite(a->factor))
        return IKBO_ERR_INVALID_ARG;
    if (a->head_dim > 1024 || a->H_q > kMaxHeads || a->H_k > kMaxHeads) return IKBO_ERR_UNSUPPORTED;
    if (a->T == 0) return IKBO_OK;
    if (!a->positions || !a->freq || (a->H_q > 0 && (!a->q || !a->q_out)) || (a->H_k > 0 && (!a->k || !a->k_out)))
        return IKBO_ERR_INVALID_ARG;
    const unsigned elt = a->dtype == IKBO_DTYPE_F32 ? 4 : 2;
    if (!aligned4(a->positions) || !aligned(a->freq, 8) || !aligned(a->q, elt) || !aligned(a->q_out, elt) ||
        !aligned(a->k, elt) || !aligned(a->k_out, elt))
        return IKBO_ERR_ALIGNMENT;
    if ((a->H_q > 0 && a->q == a->q_out && (a->q_token != a->q_out_token || a->q_head != a->q_out_head)) ||
        (a->H_k > 0 && a->k == a->k_out && (a->k_token != a->k_out_token || a->k_head != a->k_out_head)))
        return IKBO_ERR_INVALID_ARG;
    const hipError_t e = launch_rope(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "rope");
}

int ikbo_kv4_write(const ikbo_kv4_rows_args *a, void *stream) {
    const int st = check_rows(a);
    if (st != IKBO_OK) return st;
    if (a->T == 0) return IKBO_OK;
    if (!a->k || !a->v) return IKBO_ERR_INVALID_ARG;
    const hipError_t e = launch_kv4_write(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "kv4 write");
}

int ikbo_kv4_read(const ikbo_kv4_rows_args *a, void *stream) {
    const int st = check_rows(a);
    if (st != IKBO_OK) return st;
    if (a->T == 0 || (!a->k && !a->v)) return IKBO_OK;
    const hipError_t e = launch_kv4_read(*a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "kv4 read");
}

int64_t ikbo_kv4_attention_workspace(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages) {
    if (B_u < 1 || B_c < 0 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || L_q < 1 || max_pages < 1) return IKBO_ERR_INVALID_ARG;
    // Rows, units and page numbers are counted in 32 bits.
    if ((head_dim != 64 && head_dim != 128) || B_u > IKBO_KV_MAX_USERS || H_q > kMaxHeads ||
        (int64_t)max_pages * IKBO_KV4_PAGE > kInt || (int64_t)B_c * L_q > kInt / 4 || (int64_t)B_c * L_q * H_q > kInt / 4)
        return IKBO_ERR_UNSUPPORTED;
    return kv4_attn_layout(B_u, B_c, H_q, H_kv, L_q, head_dim, max_pages).total;
}

int ikbo_kv4_attention(const ikbo_kv4_attention_args *a, void *stream) {
    if (a == nullptr) return IKBO_ERR_INVALID_ARG;
    const int64_t need = ikbo_kv4_attention_workspace(a->B_u, a->B_c, a->H_q, a->H_kv, a->L_q, a->head_dim, a->max_pages);
    if (need < 0) return (int)need;
    if (a->num_pages < 1 || a->table_stride < a->max_pages || !(a->scale >= 0.0f) || std::isinf(a->scale)) return IKBO_ERR_INVALID_ARG;
    if ((int64_t)a->num_pages * IKBO_KV4_PAGE > kInt) return IKBO_ERR_UNSUPPORTED;
    if (a->B_c == 0) return IKBO_OK;
    if (!a->Q || !a->O || !a->tiles || !a->block_table || !a->lens || !a->status || !a->workspace || a->workspace_bytes < need ||
        (!a->map && a->B_c > a->B_u))
        return IKBO_ERR_INVALID_ARG;
    if (!aligned(a->Q, 16) || !aligned(a->O, 16) || !aligned(a->tiles, 16) || !aligned(a->workspace, 16) || !aligned4(a->block_table) ||
        !aligned4(a->lens) || !aligned4(a->map) || !aligned4(a->positions) || !aligned4(a->status))
        return IKBO_ERR_ALIGNMENT;
    for (int64_t s : {a->q_cand, a->q_head, a->q_query, a->o_cand, a->o_head, a->o_query})
        if (s % 8 != 0) return IKBO_ERR_ALIGNMENT;
    if (a->Q == a->O && ((a->B_c > 1 && a->q_cand != a->o_cand) || (a->H_q > 1 && a->q_head != a->o_head) ||
                         (a->L_q > 1 && a->q_query != a->o_query)))
        return IKBO_ERR_INVALID_ARG;   // rows would be written before others are read
    const Kv4AttnLayout w = kv4_attn_layout(a->B_u, a->B_c, a->H_q, a->H_kv, a->L_q, a->head_dim, a->max_pages);
    const float scale = a->scale > 0.0f ? a->scale : 1.0f / std::sqrt((float)a->head_dim);
    const hipError_t e = launch_kv4_attention(*a, w, scale, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "kv4 attention");
}

}  // extern "C"
