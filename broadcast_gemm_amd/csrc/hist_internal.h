// hist_internal.h -- host-side interface between the ABI of the cached user histories
// (ikbo_history.cpp) and its kernels (hist_*.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ikbo.h"

namespace ikbo {

// Record "what: <HIP error text>" for ikbo_last_error_message (ikbo_api.cpp); returns IKBO_ERR_HIP.
int hip_fail(hipError_t e, const char *what);

// Element `at` of a tensor of the given element size; NULL stays NULL.
template <class T>
T *beyond(T *p, int64_t at, int size) {
    return p ? reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(at * size)) : p;
}

// Bits of the caller's status word.
constexpr uint32_t kStMap = 1u, kStPage = 2u, kStNoPages = 4u, kStNonfinite = 8u;

hipError_t launch_kv_tables(const ikbo_kv_tables_args &a, hipStream_t s);
hipError_t launch_rope(const ikbo_rope_args &a, hipStream_t s);
hipError_t launch_kv4_write(const ikbo_kv4_rows_args &a, hipStream_t s);
hipError_t launch_kv4_read(const ikbo_kv4_rows_args &a, hipStream_t s);

// How the attention's work is cut (hist_plan.h), and the byte offsets of its workspace's parts.
struct Kv4AttnLayout {
    int R, log_blocks;
    int64_t line_most;                 // pages of work, at most
    int64_t o_share, o_work, o_perm, o_off, o_note, o_note_o, o_ml, o_part, total;
};
Kv4AttnLayout kv4_attn_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages);
hipError_t launch_kv4_attention(const ikbo_kv4_attention_args &a, const Kv4AttnLayout &w, float scale, hipStream_t s);

}  // namespace ikbo
