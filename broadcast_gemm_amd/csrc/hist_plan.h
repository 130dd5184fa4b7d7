// hist_plan.h -- how the cached attention's work is dealt to its blocks.
//
// A unit is (user, head, tile of R query rows); its work is the pages of the user's history (one, if
// the history is empty: its rows still have to be written).  All units' pages stand in one line, in the
// order user, head, tile, page, and every block takes one run of `share` pages of it: the blocks are
// even whatever the lengths are, and a unit is cut only where a run ends.  Neighbouring units share
// their K and V.
//
// A run's end that falls within a sixteenth of a run of a unit's edge moves to that edge: a cut costs writing and
// joining two pieces (260 KB at 256 rows of head 128), a move makes runs uneven, by an eighth at most.  1080 units of
// 13 to 16 pages in 256 runs, us with the join: 212 where a 128th moves, 204 with a sixteenth, 209 with an eighth.
//
// A block leaves at most two partial results: one of the unit that its run begins inside (slot 2 b),
// one of a unit that begins in its run and goes on after it (slot 2 b + 1).  So the pieces of a unit
// whose pages are [from, to) of the line are slot 2 b0 + 1 of the block b0 = from / share and the
// slots 2 b of the blocks after it up to (to - 1) / share: nothing about them is stored.
//
// A block in whose run a cut unit begins leaves a note of it for the launch that joins the pieces: how
// many there are, and where the rows of O stand.
//
// The line is described by the prefix sums over the users of their pages of work.  For up to 256 users
// and 1024 candidates every block of the narrow kernel forms them in LDS (2 us); beyond that, and for the
// wide kernel, whose blocks come back to other users' candidates too often to list them again each time,
// a launch of one block does (6 us and more).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hist_internal.h"

namespace ikbo {

constexpr int kPage = IKBO_KV4_PAGE;
constexpr int kPrep = 1024;                            // threads of the grouping block
constexpr int kPer = IKBO_KV_MAX_USERS / kPrep;        // users per thread of it
constexpr int kSmallUsers = 256, kSmallCands = 1024;   // plans that every block forms for itself

struct AttnArgs {
    const uint16_t *Q;
    uint16_t *O;
    const char *tiles;
    const int32_t *table, *lens, *map, *positions;
    uint32_t *status;
    int64_t *share, *work;            // [1], [B_u + 1] in the workspace
    int32_t *perm, *off;              // [B_c], [B_u + 1]
    int2 *note;                       // [blocks]: pieces (0: no cut unit begins here) and live rows
    int64_t *note_o;                  // [blocks][R]: the rows' places in O
    float2 *ml;                       // [2 * blocks][R]: maximum and sum of a partial row
    float *part;                      // [2 * blocks][R][head_dim]
    int64_t q_cand, q_head, q_query, o_cand, o_head, o_query, table_stride;
    int B_u, B_c, H_kv, G, L_q, max_pages, num_pages;
    int R, log_blocks;                // rows per unit, log2 of the blocks that share the work
    float scale_log2;
};

__device__ __forceinline__ int clamp_len(int len, int max_pages) { return min(max(len, 0), max_pages * kPage); }
__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }
__device__ __forceinline__ int64_t share_of(int64_t work, int log_blocks) {
    const int64_t s = (work + (1ll << log_blocks) - 1) >> log_blocks;
    return s > 1 ? s : 1;
}

// Runs' ends move by this much at most.
__device__ __forceinline__ int64_t near_of(int64_t share) { return share >> 4; }
// x / y for 0 <= x, 0 < y: in 32 bits where they do (a quotient in 64 takes 150 instructions).
__device__ __forceinline__ int64_t over(int64_t x, int64_t y) {
    return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}

// Exclusive scan over a wave.
template <class T>
__device__ __forceinline__ T wave_before(T v, T *total) {
    const int lane = (int)threadIdx.x & 63;
    T x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const T o = __shfl_up(x, d);
        if (lane >= d) x += o;
    }
    *total = __shfl(x, 63);
    return x - v;
}

// Largest u in [0, n) with base[u] <= x: the owner of x (users with nothing share their successor's
// base and are skipped).  64 entries at a time, one per lane.
template <class T>
__device__ __forceinline__ int owner_of(const T *base, int n, T x) {
    const int lane = (int)threadIdx.x & 63;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lane * step;
        const int k = __popcll(__ballot(i < n && base[lo + (i < n ? i : 0)] <= x)) - 1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

struct SmallPlan {
    int64_t work[kSmallUsers + 1];
    int cnt[kSmallUsers], pages[kSmallUsers];
    uint16_t map[kSmallCands];        // 0xFFFF: no user
    uint16_t list[kSmallCands];       // the candidates of user `listed`, ascending
    int listed, bad;
};
template <bool SMALL>                 // otherwise the plan stands in the workspace
using PlanLds = typename std::conditional<SMALL, SmallPlan, int>::type;

struct User {
    int u, len, pages, n_rows, tiles, cand0;
    int64_t from, to;                 // its pages in the line
};

template <bool SMALL, int NTH>
struct Plan {
    const AttnArgs &a;
    SmallPlan *sm;
    const int64_t *work;
    int64_t share;

    __device__ __forceinline__ Plan(const AttnArgs &a_, PlanLds<SMALL> &lds) : a(a_), sm(reinterpret_cast<SmallPlan *>(&lds)) {
        if constexpr (!SMALL) {
            work = a.work;
            share = a.share[0];
        } else {
            work = sm->work;
            form();
        }
    }

    __device__ __forceinline__ int tiles_of(int n_rows) const { return (n_rows + a.R - 1) / a.R; }

    __device__ __forceinline__ void form() {
        const int tid = (int)threadIdx.x, lane = tid & 63, B = a.B_u;
        constexpr int PER = kSmallUsers / 64;
        const int per = (B + 63) / 64;
        int len[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) len[e] = e < per && lane * per + e < B ? a.lens[lane * per + e] : 0;
        for (int u = tid; u < B; u += NTH) sm->cnt[u] = a.map ? 0 : u < a.B_c;
        if (tid == 0) { sm->listed = -1; sm->bad = 0; }
        __syncthreads();
        if (a.map)
            for (int b = tid; b < a.B_c; b += NTH) {
                const int u = a.map[b];
                const bool valid = u >= 0 && u < B;
                sm->map[b] = valid ? (uint16_t)u : (uint16_t)0xFFFF;
                if (valid) atomicAdd(&sm->cnt[u], 1);
                else if (u != -1) sm->bad = kStMap;
            }
        __syncthreads();
        // Every wave alike: a lane holds `per` consecutive users.
        int64_t w[PER], sum_w = 0, all_w;
        bool wrong = false;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int u = lane * per + e;
            const int rows = e < per && u < B ? sm->cnt[u] * a.L_q * a.G : 0;
            wrong = wrong || len[e] < 0 || len[e] > a.max_pages * kPage;
            const int pages = max(1, pages_of(clamp_len(len[e], a.max_pages)));
            if (tid < 64 && e < per && u < B) sm->pages[u] = pages;
            w[e] = (int64_t)tiles_of(rows) * a.H_kv * pages;
            sum_w += w[e];
        }
        int64_t at_w = wave_before(sum_w, &all_w);
        share = share_of(all_w, a.log_blocks);
        if (tid < 64) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int u = lane * per + e;
                if (e < per && u < B) {
                    sm->work[u] = at_w;
                    at_w += w[e];
                }
            }
            if (lane == 0) sm->work[B] = all_w;
        }
        const bool any = __ballot(wrong) != 0;
        __syncthreads();
        if (blockIdx.x == 0 && tid == 0 && (any || sm->bad)) atomicOr(a.status, (any ? kStPage : 0u) | (uint32_t)sm->bad);
    }

    __device__ __forceinline__ int pages_of_user(int u) const {
        if constexpr (SMALL) return sm->pages[u];
        else return max(1, pages_of(clamp_len(a.lens[u], a.max_pages)));
    }

    // The whole block comes here with the same u: its candidates become known (SMALL).
    __device__ __forceinline__ User enter(int u) {
        User x;
        x.u = u;
        x.from = work[u];
        x.to = work[u + 1];
        x.len = clamp_len(a.lens[u], a.max_pages);
        x.pages = max(1, pages_of(x.len));
        if constexpr (SMALL) {
            x.cand0 = 0;
            x.n_rows = sm->cnt[u] * a.L_q * a.G;
            if (sm->listed != u) {
                __syncthreads();   // every wave has read `listed` and is done with the old list
                if (threadIdx.x < 64) {
                    const int lane = (int)threadIdx.x;
                    if (!a.map) sm->list[0] = (uint16_t)u;   // candidate u; every lane writes the same
                    else {
                        int at = 0;
                        for (int b0 = 0; b0 < a.B_c; b0 += 64) {
                            const bool mine = b0 + lane < a.B_c && sm->map[b0 + lane] == u;
                            const uint64_t m = __ballot(mine);
                            if (mine) sm->list[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(b0 + lane);
                            at += __popcll(m);
                        }
                    }
                    if (lane == 0) sm->listed = u;
                }
                __syncthreads();
            }
        } else {
            x.cand0 = a.off[u];
            x.n_rows = (a.off[u + 1] - x.cand0) * a.L_q * a.G;
        }
        x.tiles = tiles_of(x.n_rows);
        return x;
    }
    __device__ __forceinline__ int cand(const User &x, int rank) const {
        if constexpr (SMALL) return sm->list[rank];
        else return a.perm[x.cand0 + rank];
    }
    // Row r of the user (candidate, query, head of the group) of key/value head h.
    __device__ __forceinline__ void row(const User &x, int h, int r, int &cnd, int &l, int &hq) const {
        const int per = a.L_q * a.G, rank = r / per, rest = r - rank * per;
        cnd = cand(x, rank);
        l = rest / a.G;
        hq = h * a.G + rest - l * a.G;
    }
};

}  // namespace ikbo
