// ikbo_training.cpp -- the C ABI of attention's training and of dropout declared in include/ikbo.h: argument checks,
// the layout of the work, then a few launches on the caller's stream with the caller's buffers.
#include "ikbo.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "train_internal.h"

using namespace ikbo;

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr int64_t kInt = std::numeric_limits<int32_t>::max();
constexpr int64_t kMaxToken = 1 << 24;   // elements from token to token
constexpr int kMaxHeads = 4096, kThreads = 512, kCus = 256;

// Probability as whole steps of 1 / of; 0 and `of` only for probabilities of 0 and 1.
int steps(double p, int of) { return (int)std::nearbyint(p * of); }
bool probability(double p, int of) { return p == 0.0 || (p > 0.0 && p < 1.0 && steps(p, of) > 0 && steps(p, of) < of); }

int check_shape(int B_u, int B_c, int H_q, int H_kv, int L_q, int L_kv, int head_dim) {
    if (B_u < 1 || B_c < 0 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || L_q < 1 || L_kv < 1 || head_dim < 1) return IKBO_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || B_u > IKBO_KV_MAX_USERS || H_q > kMaxHeads || L_kv > kInt / 4 || B_c > kInt / 4 ||
        (int64_t)B_c * L_q > kInt / 4 || (int64_t)B_c * L_q * H_q > kInt / 4)
        return IKBO_ERR_UNSUPPORTED;   // rows and keys are counted in 32 bits
    const TrainLayout w = train_layout(B_u, B_c, H_q, H_kv, L_q, L_kv, head_dim, true);
    // Threads of one launch are counted in 32 bits.
    const int64_t most = std::max((int64_t)w.tiles * w.splits, (int64_t)w.chunks * ((L_kv + keys_of(head_dim) - 1) / keys_of(head_dim))) * H_kv;
    return most + 64 > kInt / kThreads ? IKBO_ERR_UNSUPPORTED : IKBO_OK;
}

int check(const ikbo_attention_args *a, bool backward) {
    if (a == nullptr) return IKBO_ERR_INVALID_ARG;
    const int64_t need = ikbo_attention_workspace(a->B_u, a->B_c, a->H_q, a->H_kv, a->L_q, a->L_kv, a->head_dim, backward);
    if (need < 0) return (int)need;
    if (!(a->scale >= 0.0f) || std::isinf(a->scale) || !probability(a->dropout, 256)) return IKBO_ERR_INVALID_ARG;
    const int64_t strides[] = {a->q_cand, a->q_head, a->q_query, a->k_user, a->k_head, a->k_token, a->v_user, a->v_head, a->v_token,
                               a->o_cand, a->o_head, a->o_query, a->do_cand, a->do_head, a->do_query, a->dq_cand, a->dq_head, a->dq_query,
                               a->dk_user, a->dk_head, a->dk_token, a->dv_user, a->dv_head, a->dv_token};
    for (int i = 0; i < (backward ? 24 : 12); ++i)
        if (strides[i] < 0) return IKBO_ERR_INVALID_ARG;
    for (int i = 0; i < (backward ? 24 : 12); ++i)
        if (strides[i] % 8 != 0) return IKBO_ERR_ALIGNMENT;
    if (a->k_token > kMaxToken || a->v_token > kMaxToken) return IKBO_ERR_UNSUPPORTED;
    const bool rows = a->B_c > 0;
    if (!a->status || !a->workspace || a->workspace_bytes < need || (a->dropout > 0 && !a->rng)) return IKBO_ERR_INVALID_ARG;
    if (rows && (!a->Q || !a->K || !a->V || !a->O || !a->lse || !a->map)) return IKBO_ERR_INVALID_ARG;
    if (backward && (!a->K || !a->V || !a->dK || !a->dV || (rows && (!a->dO || !a->dQ)))) return IKBO_ERR_INVALID_ARG;
    for (const void *p : {a->Q, a->K, a->V, (const void *)a->O, (const void *)a->workspace})
        if (!aligned(p, 16)) return IKBO_ERR_ALIGNMENT;
    if (backward)
        for (const void *p : {a->dO, (const void *)a->dQ, (const void *)a->dK, (const void *)a->dV})
            if (!aligned(p, 16)) return IKBO_ERR_ALIGNMENT;
    for (const void *p : {(const void *)a->lse, (const void *)a->map, (const void *)a->lens, (const void *)a->positions, (const void *)a->status})
        if (!aligned(p, 4)) return IKBO_ERR_ALIGNMENT;
    return aligned(a->rng, 8) ? IKBO_OK : IKBO_ERR_ALIGNMENT;
}

TrainArgs args_of(const ikbo_attention_args &a, const TrainLayout &w) {
    TrainArgs t{};
    char *ws = static_cast<char *>(a.workspace);
    const auto bf16 = [](const void *p) { return static_cast<const uint16_t *>(p); };
    t.Q = bf16(a.Q); t.K = bf16(a.K); t.V = bf16(a.V); t.dO = bf16(a.dO);
    t.O = static_cast<uint16_t *>(a.O); t.lse = a.lse;
    t.dQ = static_cast<uint16_t *>(a.dQ); t.dK = static_cast<uint16_t *>(a.dK); t.dV = static_cast<uint16_t *>(a.dV);
    t.map = a.map; t.lens = a.lens; t.positions = a.positions; t.rng = a.rng; t.status = a.status;
    t.perm = reinterpret_cast<int32_t *>(ws + w.o_perm);
    t.tile = reinterpret_cast<TileEntry *>(ws + w.o_tile);
    t.chunk = reinterpret_cast<ChunkEntry *>(ws + w.o_chunk);
    t.joins = reinterpret_cast<int4 *>(ws + w.o_joins);
    t.notes = reinterpret_cast<RowNotes *>(ws + w.o_notes);
    t.part = reinterpret_cast<float *>(ws + w.o_part);
    t.ml = reinterpret_cast<float2 *>(ws + w.o_ml);
    t.part_dk = reinterpret_cast<float *>(ws + w.o_dk);
    t.part_dv = reinterpret_cast<float *>(ws + w.o_dv);
    t.q_cand = a.q_cand; t.q_head = a.q_head; t.q_query = a.q_query;
    t.k_user = a.k_user; t.k_head = a.k_head; t.k_token = a.k_token;
    t.v_user = a.v_user; t.v_head = a.v_head; t.v_token = a.v_token;
    t.o_cand = a.o_cand; t.o_head = a.o_head; t.o_query = a.o_query;
    t.do_cand = a.do_cand; t.do_head = a.do_head; t.do_query = a.do_query;
    t.dq_cand = a.dq_cand; t.dq_head = a.dq_head; t.dq_query = a.dq_query;
    t.dk_user = a.dk_user; t.dk_head = a.dk_head; t.dk_token = a.dk_token;
    t.dv_user = a.dv_user; t.dv_head = a.dv_head; t.dv_token = a.dv_token;
    t.B_u = a.B_u; t.B_c = a.B_c; t.H_q = a.H_q; t.H_kv = a.H_kv; t.G = a.H_q / a.H_kv; t.L_q = a.L_q; t.L_kv = a.L_kv;
    t.splits = w.splits; t.split_keys = w.split_keys; t.tiles = w.tiles;
    t.chunk_rows = w.chunk_rows; t.chunks = w.chunks; t.slots = w.slots; t.n_joins = w.joins; t.n_notes = w.notes;
    // Blocks for the rows of padding: one for each 256 KB of output (1024 threads; 256 in calls without the grouping).
    t.pads = (int)std::clamp<int64_t>((int64_t)a.B_c * a.H_q * a.L_q * a.head_dim >> 17, 1, 64);
    t.scale = a.scale > 0.0f ? a.scale : 1.0f / std::sqrt((float)a.head_dim);
    t.scale_log2 = (float)(t.scale * 1.4426950408889634);
    t.edge = (uint32_t)steps(a.dropout, 256);
    t.keep = (float)(256.0 / (256 - (int)t.edge));
    return t;
}

}  // namespace

namespace ikbo {

TrainLayout train_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int L_kv, int head_dim, bool backward) {
    TrainLayout w{};
    const int64_t rows = (int64_t)B_c * L_q * (H_q / H_kv);   // of one shared head, over all users
    w.tiles = (int)(rows / kTileRows + std::min(B_u, B_c));
    // Fewer blocks than CUs: the keys are cut, into four stages at least (48 candidates of 2 users with 32000 tokens: 28 us, 614
    // uncut; 50 candidates of 3 users with 200 tokens stay whole).
    const int64_t units = std::max<int64_t>((int64_t)w.tiles * H_kv, 1);
    w.splits = units >= kCus ? 1 : (int)std::min<int64_t>((2 * kCus + units - 1) / units, (L_kv + 255) / 256);
    w.split_keys = ((L_kv + w.splits - 1) / w.splits + 63) / 64 * 64;
    w.splits = (L_kv + w.split_keys - 1) / w.split_keys;
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    // Few candidates: the blocks find their places themselves, which saves the launch of the grouping.  Microseconds with the
    // launch and without: a forward of 4 users' 8 candidates 12.9 and 9.3, of 64 users' 1024 with 4096 rows 24.9 and 20.0.
    // Backward a user's rows are not cut there, so the bound is on what one user may have: 64 rows 20.4 and 16.5; 64 users with
    // 1024 rows of 4 heads 66.9 and 61.8, 4 users with 1024 47.2 and 42.1; but one user with 512 47.0 and 47.2, with 1024 46.2
    // and 70.9.
    w.local = B_u <= kLocalUsers && B_c <= kLocalCands && rows <= (backward ? std::clamp(128 * B_u, 512, 2048) : 4096);
    w.o_perm = take((int64_t)B_c * 4);
    w.o_tile = take((int64_t)w.tiles * (int64_t)sizeof(TileEntry));
    const int64_t parts = w.splits > 1 ? (int64_t)w.splits * w.tiles * H_kv * kTileRows : 0;
    w.o_part = take(parts * head_dim * 4);
    w.o_ml = take(backward ? 0 : parts * 8);
    if (backward) {
        // About twice the blocks that run at once; where the users alone make as many, a user of the average size is not cut:
        // a cut costs writing and joining its parts (70:1: 257 us and 4.6 to join; 291 and 33 without the second rule).
        const int64_t ranges = (L_kv + keys_of(head_dim) - 1) / keys_of(head_dim), at_once = kCus * 256 / keys_of(head_dim), work = rows * H_kv * ranges, whole = (int64_t)B_u * H_kv * ranges;
        int64_t each = std::max<int64_t>(work / (2 * at_once), 256);
        if (whole >= at_once * 3 / 4) each = std::max(each, rows * 5 / 4 / B_u);
        each = std::min(each, rows + 1);   // more is the same, and passes 32 bits
        w.chunk_rows = w.local ? 2048 : (int)((each + 63) / 64 * 64);   // all rows of any user
        w.chunks = w.local ? B_u : (int)(rows / w.chunk_rows + B_u);
        w.slots = rows > w.chunk_rows ? (int)(2 * rows / w.chunk_rows + 1) : 0;   // n > 1 chunks of a user are more than n / 2 full ones
        w.o_chunk = take((int64_t)w.chunks * (int64_t)sizeof(ChunkEntry));
        w.joins = std::min(B_u, w.slots / 2);
        w.o_joins = take((int64_t)w.joins * 16);
        w.notes = (int)(rows / 64 + std::min(B_u, B_c));
        w.o_notes = take((int64_t)w.notes * H_kv * (int64_t)sizeof(RowNotes));
        w.o_dk = take((int64_t)w.slots * H_kv * L_kv * head_dim * 4);
        w.o_dv = take((int64_t)w.slots * H_kv * L_kv * head_dim * 4);
    }
    w.total = std::max<int64_t>(at, 256);
    return w;
}

}  // namespace ikbo

extern "C" {

int64_t ikbo_attention_workspace(int B_u, int B_c, int H_q, int H_kv, int L_q, int L_kv, int head_dim, int backward) {
    const int st = check_shape(B_u, B_c, H_q, H_kv, L_q, L_kv, head_dim);
    return st != IKBO_OK ? st : train_layout(B_u, B_c, H_q, H_kv, L_q, L_kv, head_dim, backward != 0).total;
}

int ikbo_attention_forward(const ikbo_attention_args *a, void *stream) {
    const int st = check(a, false);
    if (st != IKBO_OK || a->B_c == 0) return st;
    const TrainLayout w = train_layout(a->B_u, a->B_c, a->H_q, a->H_kv, a->L_q, a->L_kv, a->head_dim, false);
    const TrainArgs t = args_of(*a, w);
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = w.local ? hipSuccess : launch_train_prep(t, false, a->head_dim, s);
    if (e != hipSuccess) return hip_fail(e, "attention grouping");
    e = launch_train_forward(t, w, a->head_dim, s);
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "attention forward");
}

int ikbo_attention_backward(const ikbo_attention_args *a, void *stream) {
    const int st = check(a, true);
    if (st != IKBO_OK) return st;
    const TrainLayout w = train_layout(a->B_u, a->B_c, a->H_q, a->H_kv, a->L_q, a->L_kv, a->head_dim, true);
    const TrainArgs t = args_of(*a, w);
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = w.local ? hipSuccess : launch_train_prep(t, true, a->head_dim, s);
    if (e != hipSuccess) return hip_fail(e, "attention grouping");
    e = launch_train_backward(t, w, a->head_dim, s);
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "attention backward");
}

int ikbo_dropout(const ikbo_dropout_args *a, void *stream) {
    if (a == nullptr || a->n < 0 || !probability(a->p, 65536) || (a->dtype != IKBO_DTYPE_BF16 && a->dtype != IKBO_DTYPE_F32)) return IKBO_ERR_INVALID_ARG;
    if (a->n == 0) return IKBO_OK;
    if (!a->x || !a->y || !a->rng) return IKBO_ERR_INVALID_ARG;
    const unsigned size = a->dtype == IKBO_DTYPE_F32 ? 4 : 2;
    if (!aligned(a->x, size) || !aligned(a->y, size) || !aligned(a->residual, size) || !aligned(a->rng, 8)) return IKBO_ERR_ALIGNMENT;
    const hipError_t e = launch_dropout(*a, (uint32_t)steps(a->p, 65536), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IKBO_OK : hip_fail(e, "dropout");
}

}  // extern "C"
