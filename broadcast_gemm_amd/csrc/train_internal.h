// train_internal.h -- host-side interface between the ABI of attention's training and dropout
// (ikbo_training.cpp) and its kernels (train_*.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ikbo.h"

namespace ikbo {

// Record "what: <HIP error text>" for ikbo_last_error_message (ikbo_api.cpp); returns IKBO_ERR_HIP.
int hip_fail(hipError_t e, const char *what);

// Bits of the caller's status word, as in the cached histories.
constexpr uint32_t kTrainStMap = 1u, kTrainStLens = 2u;

// Keys to a block of dK and dV: 8 waves or 4, of 32.  Head 128: 8 waves share the rows' staging (259 us, 4 waves 270); head 64:
// 4, two blocks of which stand on a CU (65 us, 8 waves 88; 26 users, 256 candidates of 33 queries, dropout).
constexpr int keys_of(int head_dim) { return head_dim == 128 ? 256 : 128; }
// Waves and rows of a block of the forward and of dQ.  Two blocks of 4 waves a CU: 70:1 with head 128, forward 154 us and dQ
// 220, where one of 8 waves takes 180 and 253: its waves meet at every barrier.
constexpr int kRowWaves = 4, kTileRows = 32 * kRowWaves;
constexpr int kLocalUsers = 64, kLocalCands = 1024;   // calls up to which blocks find their places for themselves
constexpr int kJoiners = 8;       // groups of lanes that add up the parts of a row

// How the work is cut, and the byte offsets of the workspace's parts.  A user's rows of one shared head are its
// candidates' queries of all heads of the group: slot * G * L_q + g * L_q + l, with the candidates in order.
struct TrainLayout {
    bool local;                        // every block finds its own place: no launch of the grouping
    int tiles;                         // tiles of rows per shared head, at most
    int splits, split_keys;            // parts of the keys, each a multiple of 64
    int chunk_rows;                    // rows to a block of dK and dV, at most
    int chunks, slots, joins;          // blocks of them per shared head and range of keys, at most; those with partial results; their users
    int notes;                         // 64 rows each, per shared head, at most
    int64_t o_perm, o_tile, o_chunk, o_joins, o_notes, o_part, o_ml, o_dk, o_dv, total;
};
TrainLayout train_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int L_kv, int head_dim, bool backward);

// A tile of rows, and a chunk of them for dK and dV; user -1 where there is none.
struct TileEntry {
    int user, row, first, rows;        // its first row; the user's candidates in perm, and rows
    int len, note, unused[2];          // tokens of the user; the notes of `row`
};
struct ChunkEntry {
    int user, note, notes, slot;       // its notes and how many; place of its partial result or -1
    int len, unused[3];
};

// What the dQ kernel notes of 64 rows of a user for the dK and dV kernel, which loads it straight into LDS.
struct RowNotes {
    const void *q[64], *dy[64];        // where they stand; a row that does not exist or sees nothing is a row of zeros
    float shift[64], D[64];            // -lse in base 2 (-inf for such a row: no weights), rowsum(dO O)
    int limit[64], row[64], head[64];  // tokens it sees, b L_q + l, h
    int most[2];                       // largest limit of each 32
    int unused[190];                   // whole KB
};
static_assert(sizeof(RowNotes) == 3 * 1024, "three loads of a wave");

struct TrainArgs {
    const uint16_t *Q, *K, *V;
    uint16_t *O;
    float *lse;
    const uint16_t *dO;
    uint16_t *dQ, *dK, *dV;
    const int32_t *map, *lens, *positions;
    const int64_t *rng;
    uint32_t *status;
    int32_t *perm;                     // [B_c] candidates by user
    TileEntry *tile;                   // [tiles]
    ChunkEntry *chunk;                 // [chunks]
    int4 *joins;                       // [slots / 2]: user, tokens, its first place among the partial results, how many; 0 of them: none
    RowNotes *notes;                   // [H_kv][notes]
    float *part;                       // partial O or dQ [splits][tiles][H_kv][tile_rows][head_dim]
    float2 *ml;                        // maximum and sum of a partial row of O, likewise
    float *part_dk, *part_dv;          // [slots][H_kv][L_kv rounded up][head_dim]
    int64_t q_cand, q_head, q_query, k_user, k_head, k_token, v_user, v_head, v_token, o_cand, o_head, o_query;
    int64_t do_cand, do_head, do_query, dq_cand, dq_head, dq_query, dk_user, dk_head, dk_token, dv_user, dv_head, dv_token;
    int B_u, B_c, H_q, H_kv, G, L_q, L_kv;
    int splits, split_keys, tiles, chunk_rows, chunks, slots, n_joins, n_notes;
    float scale, scale_log2;
    uint32_t edge;                     // weights whose byte is below it are dropped
    float keep;                        // 256 / (256 - edge)
    int pads;                          // blocks that fill the rows of padding
};

// What a launch of the grouping fills in for padding: O and lse, or dQ.
hipError_t launch_train_prep(const TrainArgs &a, bool backward, int head_dim, hipStream_t s);
hipError_t launch_train_forward(const TrainArgs &a, const TrainLayout &w, int head_dim, hipStream_t s);
hipError_t launch_train_backward(const TrainArgs &a, const TrainLayout &w, int head_dim, hipStream_t s);
// Elements whose 16 bits are below edge are dropped.
hipError_t launch_dropout(const ikbo_dropout_args &a, uint32_t edge, hipStream_t s);

}  // namespace ikbo
