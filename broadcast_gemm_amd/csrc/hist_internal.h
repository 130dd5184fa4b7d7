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
// Record `what` for ikbo_last_error_message; returns status.
int status_fail(int status, const char *what);

// Bits of the caller's status word.
constexpr uint32_t kStMap = 1u, kStPage = 2u, kStNoPages = 4u, kStNonfinite = 8u;

hipError_t launch_kv_tables(const ikbo_kv_tables_args &a, hipStream_t s);
hipError_t launch_rope(const ikbo_rope_args &a, hipStream_t s);
hipError_t launch_kv4_write(const ikbo_kv4_rows_args &a, hipStream_t s);
hipError_t launch_kv4_read(const ikbo_kv4_rows_args &a, hipStream_t s);

// Workspace of the attention: byte offsets of its parts.
struct Kv4AttnLayout {
    int rows_per_unit, units;          // query rows of one unit, and about how many units are made
    int64_t o_hdr, o_perm, o_off, o_ubase, o_pbase, o_tbase, o_ml, o_part, total;
    int64_t part_units;                // units that may leave a partial result
};
Kv4AttnLayout kv4_attn_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages);
hipError_t launch_kv4_attention(const ikbo_kv4_attention_args &a, const Kv4AttnLayout &w, float scale, hipStream_t s);

}  // namespace ikbo
