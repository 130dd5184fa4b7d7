// train_backward.hip -- the gradients of target attention (ikbo_attention_backward), probabilities recomputed.
//
// Two kernels, each with all it sums in registers, so that nothing is added up by atomics and no block waits for another:
//
// dQ: as the forward, a block takes a tile of rows against a range of keys: S^T = K Q^T, dP^T = V dO^T, P = exp(S - lse),
// dS = P (dP - D), dQ^T += K^T dS^T.  It first forms D = rowsum(dO O), which the other kernel reads.  For a row that
// sees no more than the first 128 keys D is the sum of P dP instead, formed before: with few keys the rounding of O shows
// in dP - D, and would be a third of the error.
//
// dK and dV: a wave keeps 32 keys' K and V and their gradients in registers, and the block goes over a chunk of the
// user's rows, staged in LDS 64 at a time: S = Q K^T, dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS.  Rows stand in the
// results' rows here, so P and dS are the B operands as they stand.  The weights that stay are decided with the rows
// in the lanes, as in the other kernels (one generator call for 16 tokens of a row), and the bits turned round (Turn).
// Chunks of one user are joined by a third launch, in their order.
//
// That is 7 products against the 5 that one pass needs; adding up dQ across key ranges instead would write and read 4
// bytes an element for every range.  P and dS are rounded to bf16 for their products (half a step each, as the outputs); all
// sums are float32.
//
// Measured, with the batch of the forward (15 users, 1024 candidates of 64 queries, 4 heads of 128): dQ 211 to 214 us, dK
// and dV 253 to 257, by the card: 850 and 945 TFLOP/s of their own products (3 and 4 of them).  Both stand two waves to a SIMD with nearly all 256
// registers, and are bound by that: a wave's products wait for its own exponentials and LDS reads (256 bytes a cycle, no
// conflicts), and only one other wave fills the time.  What made the difference: V in LDS for dK and dV, for two waves on
// a SIMD instead of one (921 -> 407 us); no spilled register in the loop, as a reload waits for all loads of the next
// stage (407 -> 255); operands read one step ahead between fences; rows noted once by the dQ kernel.  Half the keys a
// block there takes 270, reading two or three steps ahead 252 and 259, 64 keys a wave does not fit the registers.
// 26 users, 256 candidates of 33 queries, 8 heads of 64, dropout: 50 and 65 us.  8001 candidates, one query each, with
// positions, 16 heads on 4: 65 and 104.
#include <algorithm>

#include "train_device.h"

namespace ikbo {
namespace {

template <int HD, int WAVES, bool DROP, bool LOCAL>
__global__ void __launch_bounds__(64 * WAVES, 2) train_dq_kernel(TrainArgs a) {
    constexpr int TK = HD / 16, DT = HD / 32, STAGE = Rows<HD>::matrix(64), ROWS = 32 * WAVES;
    __shared__ __align__(16) char lds[2][2][STAGE];
    __shared__ int s_most[WAVES], s_least[WAVES];
    if constexpr (LOCAL) {
        const int pad = (int)blockIdx.x - (int)gridDim.x + a.pads;
        if (pad >= 0) {   // the last blocks
            fill_padding(a, HD, true, pad);
            return;
        }
    }
    const int unit = unit_of((int)blockIdx.x, a.tiles * a.H_kv * a.splits);
    if (unit < 0) return;   // the whole block: no barrier has run
    const auto [tile, hk, split] = tile_unit(a, unit);
    Local<64 * WAVES> local;
    __shared__ LocalLds s_local;
    TileEntry t;
    if constexpr (LOCAL) {
        local.count(a, s_local);
        t = local.tile(tile);
        if (a.splits > 1 && hk == 0 && split == 0 && threadIdx.x == 0) a.tile[tile] = t;   // for the launch that joins
    } else {
        t = a.tile[tile];
    }
    const int u = __builtin_amdgcn_readfirstlane(t.user), row0 = __builtin_amdgcn_readfirstlane(t.row);
    if (u < 0) return;
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5, j = lane & 31;
    const int n_rows = __builtin_amdgcn_readfirstlane(t.rows), len = __builtin_amdgcn_readfirstlane(t.len);

    // The first keys are on their way before the rows.
    const int key0 = split * a.split_keys;
    const uint32_t lds0 = lds_address(lds);
    KeyLoads<HD, WAVES> keys;
    keys.init(a, u, hk, lane, wv);
    auto load = [&](int st) {
        const uint32_t to = lds0 + (st & 1) * 2 * STAGE;
        keys.load_k(to, wv, key0 + 64 * st, len);
        keys.load_v(to + STAGE, wv, key0 + 64 * st, len);
    };
    load(0);
    if constexpr (LOCAL) {
        local.list(a, s_local, u);
        if (a.splits > 1 && hk == 0 && split == 0 && row0 == 0)
            for (int i = tid; i * a.G * a.L_q < n_rows; i += 64 * WAVES) a.perm[t.first + i] = s_local.list[i];
    }
    auto place = [&](int r) {
        if constexpr (LOCAL) return place_of(a, s_local.list, hk, r);
        else return place_of(a, a.perm + t.first, hk, r);
    };
    const int r = row0 + wv * 32 + j;
    const bool live = r < n_rows;
    int limit, most, least;
    uint32_t row, head;
    u32x4_t qf[TK], gf[TK];
    float shift, D;
    {
        const Place at = place(live ? r : 0);
        limit = live ? limit_of(a, at, len) : 0;
        row = (uint32_t)(at.cand * a.L_q + at.query);
        head = (uint32_t)at.head;
        const bool sees = limit > 0;   // other rows are not read: they have no gradient, whatever theirs is
        const uint16_t *q = a.Q + at.cand * a.q_cand + at.head * a.q_head + at.query * a.q_query + 8 * g;
        const uint16_t *dy = a.dO + at.cand * a.do_cand + at.head * a.do_head + at.query * a.do_query + 8 * g;
        const uint16_t *y = a.O + at.cand * a.o_cand + at.head * a.o_head + at.query * a.o_query + 8 * g;
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < TK; ++s) {
            qf[s] = sees ? *reinterpret_cast<const u32x4_t *>(q + 16 * s) : (u32x4_t){0, 0, 0, 0};
            gf[s] = sees ? *reinterpret_cast<const u32x4_t *>(dy + 16 * s) : (u32x4_t){0, 0, 0, 0};
            const u32x4_t of = sees ? *reinterpret_cast<const u32x4_t *>(y + 16 * s) : (u32x4_t){0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum = __builtin_fmaf(__builtin_bit_cast(float, of[e] << 16), __builtin_bit_cast(float, gf[s][e] << 16), sum);
                sum = __builtin_fmaf(__builtin_bit_cast(float, of[e] & 0xFFFF0000u), __builtin_bit_cast(float, gf[s][e] & 0xFFFF0000u), sum);
            }
        }
        D = sum_halves(sum);
        shift = sees ? -a.lse[((int64_t)at.cand * a.H_q + at.head) * a.L_q + at.query] * kLog2e : 0.f;
        most = limit;
        least = live ? limit : len;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        most = max(most, __shfl_xor(most, d));
        least = min(least, __shfl_xor(least, d));
    }
    most = __builtin_amdgcn_readfirstlane(most);
    least = __builtin_amdgcn_readfirstlane(least);
    if (lane == 0) {
        s_most[wv] = most;
        s_least[wv] = least;
    }
    __syncthreads();
    int end = 0, fewest = len;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        end = max(end, s_most[w]);
        fewest = min(fewest, s_least[w]);
    }
    end = min(end, key0 + a.split_keys);

    Random rnd;
    if constexpr (DROP) rnd.init(a.rng);
    f32x16_t dq[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) dq[d] = (f32x16_t)(0.f);
    Reader<HD> rd;
    rd.init(lane);
    const int stages = max(0, (end - key0 + 63) >> 6);
    landed();   // also where no stage is wanted: nothing may arrive after the block
    // P in S, and dP, of keys t0 + 8 (i / 4) + 4 g + i % 4, t0 = key0 + 64 st + 32 h.
    f32x16_t S, dP;
    auto probabilities = [&](int st, int h) {
        const char *K = lds[st & 1][0], *V = lds[st & 1][1];
        const int t0 = key0 + 64 * st + 32 * h;
        S = dP = (f32x16_t)(0.f);
        u32x4_t kf[2] = {rd.direct(K, h, 0)}, vf[2] = {rd.direct(V, h, 0)};   // a step ahead
#pragma unroll
        for (int s = 0; s < TK; ++s) {
            if (s + 1 < TK) {
                kf[(s + 1) & 1] = rd.direct(K, h, s + 1);
                vf[(s + 1) & 1] = rd.direct(V, h, s + 1);
            }
            S = mfma32(kf[s & 1], qf[s], S);
            dP = mfma32(vf[s & 1], gf[s], dP);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[i], a.scale_log2, shift));
        if constexpr (DROP) {
            const u32x4_t w = rnd.weights(t0 >> 5, g, row, head);
#pragma unroll
            for (int i = 0; i < 16; ++i) dP[i] = ((w[i >> 2] >> (8 * (i & 3))) & 255u) >= a.edge ? dP[i] * a.keep : 0.f;
        }
        if (t0 + 32 > least) {
            asm volatile("");   // stays a branch: as selects its body would be paid by every stage
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (t0 + 8 * (i >> 2) + 4 * g + (i & 3) >= limit) S[i] = 0.f;
        }
    };
    if (key0 == 0 && stages > 0 && fewest <= 128) {
        __syncthreads();
        if (stages > 1) load(1);
        landed();
        __syncthreads();
        float sum = 0.f;
#pragma unroll 1
        for (int x = 0; x < 2 * min(stages, 2); ++x) {
            probabilities(x >> 1, x & 1);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = __builtin_fmaf(S[i], dP[i], sum);
        }
        sum = sum_halves(sum);
        D = limit <= 128 ? sum : D;
    }
    for (int st = 0; st < stages; ++st) {
        landed();
        __syncthreads();   // stage st is there, and its other buffer has been read
        if (st + 1 < stages) load(st + 1);
        if (key0 + 64 * st >= most) continue;   // none of the wave's rows sees these keys
        const char *K = lds[st & 1][0];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            probabilities(st, h);
            u32x4_t pf[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) pf[i >> 3][(i >> 1) & 3] = pack_bf16x2(S[i] * (dP[i] - D), S[i + 1] * (dP[i + 1] - D));
            u32x4_t kt[2] = {rd.turned(K, 2 * h, 0)};
#pragma unroll
            for (int i = 0; i < 2 * DT; ++i) {
                if (i + 1 < 2 * DT) kt[(i + 1) & 1] = rd.turned(K, 2 * h + (i + 1) / DT, (i + 1) % DT);
                dq[i % DT] = mfma32(kt[i & 1], pf[i / DT], dq[i % DT]);
            }
        }
    }
    const Place at = place(live ? r : 0);   // again, rather than kept
    if (split == 0 && r < ((n_rows + 63) & ~63)) {
        RowNotes &x = a.notes[(int64_t)hk * a.n_notes + t.note + ((r - row0) >> 6)];
        if (g == 0) {
            const int i = r & 63;
            const bool sees = limit > 0;
            x.q[i] = sees ? (const void *)(a.Q + at.cand * a.q_cand + at.head * a.q_head + at.query * a.q_query) : kZeroRow;
            x.dy[i] = sees ? (const void *)(a.dO + at.cand * a.do_cand + at.head * a.do_head + at.query * a.do_query) : kZeroRow;
            x.shift[i] = sees ? shift : neg_inf();
            x.D[i] = D;
            x.limit[i] = limit;
            x.row[i] = at.cand * a.L_q + at.query;
            x.head[i] = at.head;
        }
        if (lane == 0) x.most[wv & 1] = most;
    }
    if (!live) return;
    if (a.splits == 1) {
        uint16_t *to = a.dQ + at.cand * a.dq_cand + at.head * a.dq_head + at.query * a.dq_query + 8 * g;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int p = 0; p < 2; ++p) *reinterpret_cast<u32x4_t *>(to + 32 * d + 16 * p) = eight_rows(dq[d], p, a.scale);
    } else {
        float *to = a.part + ((((int64_t)split * a.tiles + tile) * a.H_kv + hk) * ROWS + wv * 32 + j) * HD + 4 * g;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4_t *>(to + 32 * d + 8 * q) = (f32x4_t){dq[d][4 * q], dq[d][4 * q + 1], dq[d][4 * q + 2], dq[d][4 * q + 3]};
    }
}

// As in the forward, the parts of one row of dQ: kJoiners groups of HD / 4 lanes take every kJoiners-th each.
template <int HD>
__global__ void __launch_bounds__(256) train_dq_join_kernel(TrainArgs a) {
    constexpr int LANES = HD / 4, ROWS = 256 / LANES / kJoiners;
    __shared__ f32x4_t parts[kJoiners][ROWS][LANES];
    const int x = (int)threadIdx.x % LANES, row = (int)threadIdx.x / LANES % ROWS, part = (int)threadIdx.x / LANES / ROWS;
    const int64_t i = (int64_t)blockIdx.x * ROWS + row;
    const int in_tile = (int)(i % kTileRows), hk = (int)(i / kTileRows % a.H_kv), tile = (int)(i / kTileRows / a.H_kv);
    const TileEntry t = a.tile[min(tile, a.tiles - 1)];
    const int r = t.row + in_tile;
    const bool live = tile < a.tiles && t.user >= 0 && r < t.rows;
    const int64_t row0 = ((int64_t)tile * a.H_kv + hk) * kTileRows + in_tile, step = (int64_t)a.tiles * a.H_kv * kTileRows;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    if (live) {
#pragma unroll 4
        for (int s = part; s < a.splits; s += kJoiners) o += *reinterpret_cast<const f32x4_t *>(a.part + (row0 + s * step) * HD + 4 * x);
    }
    parts[part][row][x] = o;
    __syncthreads();
    if (part > 0 || !live) return;
#pragma unroll
    for (int y = 1; y < kJoiners; ++y) o += parts[y][row][x];
    const Place p = place_of(a, a.perm + t.first, hk, r);
    *reinterpret_cast<u32x2_t *>(a.dQ + p.cand * a.dq_cand + p.head * a.dq_head + p.query * a.dq_query + 4 * x) =
        (u32x2_t){pack_bf16x2(o[0] * a.scale, o[1] * a.scale), pack_bf16x2(o[2] * a.scale, o[3] * a.scale)};
}

template <int HD, int WAVES, bool DROP, bool LOCAL>
__global__ void __launch_bounds__(64 * WAVES, 2) train_dkv_kernel(TrainArgs a) {
    constexpr int TK = HD / 16, DT = HD / 32, STAGE = Rows<HD>::matrix(64), KEYS = 32 * WAVES, N = 64 * HD / 8 / (64 * WAVES);
    constexpr bool V_LDS = HD == 128;   // V stays in LDS: 32 registers less, which lets two waves stand on a SIMD
    __shared__ __align__(16) char lds[2][2][STAGE], v_lds[V_LDS ? Rows<HD>::matrix(KEYS) : 16];
    __shared__ __align__(16) RowNotes notes[3];
    __shared__ int s_stages[WAVES];
    const int ranges = (a.L_kv + KEYS - 1) / KEYS;
    const int unit = unit_of((int)blockIdx.x, a.chunks * a.H_kv * ranges);
    if (unit < 0) return;   // the whole block: no barrier has run
    const int range = unit % ranges, hk = unit / ranges % a.H_kv, c = unit / ranges / a.H_kv;   // neighbours share rows
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5, j = lane & 31;
    ChunkEntry ch;
    if constexpr (LOCAL) {
        __shared__ LocalLds s_local;
        Local<64 * WAVES> local;
        local.count(a, s_local);
        ch = local.chunk(c);
    } else {
        ch = a.chunk[c];
    }
    const int u = __builtin_amdgcn_readfirstlane(ch.user), len = __builtin_amdgcn_readfirstlane(ch.len);
    if (u < 0) return;
    const int key0 = range * KEYS + wv * 32, slot = __builtin_amdgcn_readfirstlane(ch.slot);

    const int token = turned_token(j);   // of each 32 keys, the one in this lane
    Random rnd;
    Turn<!V_LDS> turn;
    if constexpr (DROP) {
        rnd.init(a.rng);
        turn.lane = lane;
    }
    // Keys behind the history and users without candidates: zeros, and nothing is read.
    int stages = range * KEYS < len ? __builtin_amdgcn_readfirstlane(ch.notes) : 0;
    u32x4_t kf[TK], vf[V_LDS ? 1 : TK];
    f32x16_t dk[DT], dv[DT];
    {
        const int t = key0 + token;
        const uint16_t *k = a.K + u * a.k_user + hk * a.k_head + t * a.k_token + 8 * g;
        const uint16_t *v = a.V + u * a.v_user + hk * a.v_head + t * a.v_token + 8 * g;
#pragma unroll
        for (int s = 0; s < TK; ++s) {
            kf[s] = stages > 0 && t < len ? *reinterpret_cast<const u32x4_t *>(k + 16 * s) : (u32x4_t){0, 0, 0, 0};
            if constexpr (!V_LDS) vf[s] = stages > 0 && t < len ? *reinterpret_cast<const u32x4_t *>(v + 16 * s) : (u32x4_t){0, 0, 0, 0};
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) dk[d] = dv[d] = (f32x16_t)(0.f);
    }
    const char *V = v_lds + Rows<HD>::matrix(32) * wv;
    if (V_LDS && stages > 0) {   // each wave its own keys
        const uint16_t *v = a.V + u * a.v_user + hk * a.v_head;
#pragma unroll
        for (int i = 0; i < 32 * HD / 8 / 64; ++i) {
            const int p = i * 64 + lane, row = p / Rows<HD>::CHUNKS, chunk = ((p % Rows<HD>::CHUNKS) ^ Rows<HD>::number(row)) * 16;
            const int t = key0 + turned_token(row);
            load_to_lds(t < len ? reinterpret_cast<const char *>(v + t * a.v_token) + chunk : reinterpret_cast<const char *>(kZeroRow) + chunk,
                        lds_address(V) + i * Rows<HD>::GROUP);
        }
    }
    Reader<HD> rd;
    rd.init(lane);
    const uint32_t lds0 = lds_address(lds);
    const char *from_notes = reinterpret_cast<const char *>(a.notes + (int64_t)hk * a.n_notes + __builtin_amdgcn_readfirstlane(ch.note));
    auto load_notes = [&](int n) {
#pragma unroll
        for (int i = 0; i < 3; ++i) load_to_lds(from_notes + (int64_t)n * (int)sizeof(RowNotes) + 1024 * i, 16 * lane, lds_address(&notes[n % 3]) + 1024 * i);
    };
    auto load = [&](int st) {
        const RowNotes &x = notes[st % 3];
        const uint32_t to = lds0 + (st & 1) * 2 * STAGE;
        int p0 = (int)threadIdx.x;
        if constexpr (V_LDS) asm volatile("" : "+v"(p0));   // places formed here: kept, they would be spilled
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = i * 64 * WAVES + p0, row = p / Rows<HD>::CHUNKS;
            const int chunk = ((p % Rows<HD>::CHUNKS) ^ Rows<HD>::number(row)) * 16;
            load_to_lds(static_cast<const char *>(x.q[row]) + chunk, to + (i * WAVES + wv) * Rows<HD>::GROUP);
            load_to_lds(static_cast<const char *>(x.dy[row]) + chunk, to + STAGE + (i * WAVES + wv) * Rows<HD>::GROUP);
        }
    };
    if (a.positions) {   // rows stand about in the order of their positions, far ones first: up to the last stage that sees the block's keys
        const RowNotes *x = a.notes + (int64_t)hk * a.n_notes + ch.note;
        int mine = 0;
        for (int st = tid; st < stages; st += 64 * WAVES)
            if (max(x[st].most[0], x[st].most[1]) > range * KEYS) mine = st + 1;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) mine = max(mine, __shfl_xor(mine, d));
        if (lane == 0) s_stages[wv] = mine;
        __syncthreads();
        stages = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) stages = max(stages, s_stages[w]);
        stages = __builtin_amdgcn_readfirstlane(stages);
    }
    if (wv == 0 && stages > 0) load_notes(0);
    if (wv == 0 && stages > 1) load_notes(1);
    landed();   // also where no stage is wanted: nothing may arrive after the block
    if (stages > 0) {
        __syncthreads();
        load(0);
    }
    for (int st = 0; st < stages; ++st) {
        landed();
        __syncthreads();   // stage st and the notes of the next are there, and the other buffer has been read
        if (st + 1 < stages) load(st + 1);
        if (wv == 0 && st + 2 < stages) load_notes(st + 2);
        const RowNotes &x = notes[st % 3];
        int at = (int)threadIdx.x & 63;
        if constexpr (V_LDS) asm volatile("" : "+v"(at));
        const int limit = x.limit[at];
        if (!__ballot(limit > key0)) continue;   // no row sees the wave's keys
        const bool partly = __ballot(limit < key0 + 32) != 0;
        const char *Q = lds[st & 1][0], *Y = lds[st & 1][1];
        // What stays of the lane's token, of the rows 32 h.
        auto staying = [&](int h) {
            return turn.rows(rnd.weights(key0 >> 5, g, (uint32_t)x.row[32 * h + j], (uint32_t)x.head[32 * h + j]), a.edge) >> (4 * g);
        };
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const float *shifts = x.shift + 32 * h + 4 * g, *Ds = x.D + 32 * h + 4 * g;
            const int *limits = x.limit + 32 * h + 4 * g;
            f32x16_t S, dP;
            u32x4_t pf[2], sf[2];
            uint32_t stays;
            S = dP = (f32x16_t)(0.f);
            // Weights and gradients of the scores of rows 8 q + 4 g + e.
            auto four = [&](int q, const f32x4_t &shift, const f32x4_t &D) {
                float p[4], ds[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[4 * q + e], a.scale_log2, shift[e]));
                if (partly) {
                    asm volatile("");   // stays a branch: as selects its body would be paid by every stage
                    const u32x4_t limit = *reinterpret_cast<const u32x4_t *>(limits + 8 * q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = key0 + token < (int)limit[e] ? p[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float dp = dP[4 * q + e];
                    const bool stay = !DROP || (stays >> (8 * q + e) & 1);
                    if constexpr (DROP) dp = stay ? dp * a.keep : 0.f;
                    ds[e] = p[e] * (dp - D[e]);
                    if constexpr (DROP) p[e] = stay ? p[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pf[q >> 1][2 * (q & 1) + e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
                    sf[q >> 1][2 * (q & 1) + e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
                }
            };
            if constexpr (!V_LDS) {
#pragma unroll
                for (int s = 0; s < TK; ++s) {
                    S = mfma32(rd.direct(Q, h, s), kf[s], S);
                    dP = mfma32(rd.direct(Y, h, s), vf[s], dP);
                }
                if constexpr (DROP) stays = staying(h);
#pragma unroll
                for (int q = 0; q < 4; ++q) four(q, *reinterpret_cast<const f32x4_t *>(shifts + 8 * q), *reinterpret_cast<const f32x4_t *>(Ds + 8 * q));
#pragma unroll
                for (int i = 0; i < 2 * DT; ++i) {
                    dv[i % DT] = mfma32(rd.turned(Y, 2 * h + i / DT, i % DT), pf[i / DT], dv[i % DT]);
                    dk[i % DT] = mfma32(rd.turned(Q, 2 * h + i / DT, i % DT), sf[i / DT], dk[i % DT]);
                }
            } else {
                // Operands are read one step ahead of their products, and the first of a part before the part before it is
                // over.  The fences keep the compiler from reading all of them first, for which it would spill: the load of
                // a spilled register would wait for the next stage's.  Two or three steps ahead made no difference (252, 259 us).
                u32x4_t qf[2], yf[2], vl[2], yt[2], qt[2];
                auto operands = [&](int s) {
                    qf[s & 1] = rd.direct(Q, h, s);
                    yf[s & 1] = rd.direct(Y, h, s);
                    vl[s & 1] = rd.direct(V, 0, s);
                };
                auto turned = [&](int i) {
                    yt[i & 1] = rd.turned(Y, 2 * h + i / DT, i % DT);
                    qt[i & 1] = rd.turned(Q, 2 * h + i / DT, i % DT);
                };
                f32x4_t shift[2], D[2];
                auto rows = [&](int q) {
                    shift[q & 1] = *reinterpret_cast<const f32x4_t *>(shifts + 8 * q);
                    D[q & 1] = *reinterpret_cast<const f32x4_t *>(Ds + 8 * q);
                };
                operands(0);
#pragma unroll
                for (int s = 0; s < TK; ++s) {
                    if (s + 1 < TK) operands(s + 1);
                    else if (!DROP) rows(0);
                    S = mfma32(qf[s & 1], kf[s], S);
                    dP = mfma32(yf[s & 1], vl[s & 1], dP);
                    fence();
                }
                if constexpr (DROP) {
                    stays = staying(h);
                    fence();
                    rows(0);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q < 3) rows(q + 1);
                    else turned(0);
                    four(q, shift[q & 1], D[q & 1]);
                    fence();
                }
#pragma unroll
                for (int i = 0; i < 2 * DT; ++i) {
                    if (i + 1 < 2 * DT) turned(i + 1);
                    dv[i % DT] = mfma32(yt[i & 1], pf[i / DT], dv[i % DT]);
                    dk[i % DT] = mfma32(qt[i & 1], sf[i / DT], dk[i % DT]);
                    fence();
                }
            }
        }
    }
    const int t = key0 + token;
    if (t < a.L_kv) {
        if (slot < 0) {
            const float by = t < len ? 1.f : 0.f;   // what a key behind the history has gathered is no gradient
            uint16_t *k = a.dK + u * a.dk_user + hk * a.dk_head + t * a.dk_token + 8 * g, *v = a.dV + u * a.dv_user + hk * a.dv_head + t * a.dv_token + 8 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const u32x4_t x = eight_rows(dk[d], p, a.scale), y = eight_rows(dv[d], p, a.keep), zero = {0, 0, 0, 0};
                    *reinterpret_cast<u32x4_t *>(k + 32 * d + 16 * p) = by > 0.f ? x : zero;
                    *reinterpret_cast<u32x4_t *>(v + 32 * d + 16 * p) = by > 0.f ? y : zero;
                }
        } else {
            const int64_t row = ((int64_t)slot * a.H_kv + hk) * a.L_kv + t;
            float *k = a.part_dk + row * HD + 4 * g, *v = a.part_dv + row * HD + 4 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    *reinterpret_cast<f32x4_t *>(k + 32 * d + 8 * q) = (f32x4_t){dk[d][4 * q], dk[d][4 * q + 1], dk[d][4 * q + 2], dk[d][4 * q + 3]};
                    *reinterpret_cast<f32x4_t *>(v + 32 * d + 8 * q) = (f32x4_t){dv[d][4 * q], dv[d][4 * q + 1], dv[d][4 * q + 2], dv[d][4 * q + 3]};
                }
        }
    }
}

// dK and dV of 16 keys from the chunks of their user, in the order of the chunks; HD / 4 lanes a key.  Bound by reading the
// parts: 8 us for 23 users, two thirds of 8001 candidates with one.
template <int HD>
__global__ void __launch_bounds__(256) train_dkv_join_kernel(TrainArgs a) {
    constexpr int LANES = HD / 4;
    const int blocks = (a.L_kv + 15) / 16, x = (int)threadIdx.x % LANES;
    const int4 join = a.joins[(int)blockIdx.x / (blocks * a.H_kv)];   // user, its tokens, first place, places
    const int u = join.x, hk = (int)blockIdx.x / blocks % a.H_kv;
    if (join.w == 0) return;
    for (int t = (int)blockIdx.x % blocks * 16 + (int)threadIdx.x / LANES, end = min(a.L_kv, t / 16 * 16 + 16); t < end; t += 256 / LANES) {
        f32x4_t k = {0.f, 0.f, 0.f, 0.f}, v = {0.f, 0.f, 0.f, 0.f};
        if (t < join.y) {
#pragma unroll 4
            for (int c = 0; c < join.w; ++c) {
                const int64_t row = ((int64_t)(join.z + c) * a.H_kv + hk) * a.L_kv + t;
                k += *reinterpret_cast<const f32x4_t *>(a.part_dk + row * HD + 4 * x);
                v += *reinterpret_cast<const f32x4_t *>(a.part_dv + row * HD + 4 * x);
            }
            k *= a.scale;
            v *= a.keep;
        }
        *reinterpret_cast<u32x2_t *>(a.dK + u * a.dk_user + hk * a.dk_head + t * a.dk_token + 4 * x) = (u32x2_t){pack_bf16x2(k[0], k[1]), pack_bf16x2(k[2], k[3])};
        *reinterpret_cast<u32x2_t *>(a.dV + u * a.dv_user + hk * a.dv_head + t * a.dv_token + 4 * x) = (u32x2_t){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

template <int HD, int WAVES, int KW>
hipError_t launch(const TrainArgs &a, bool local, hipStream_t s) {
    static_assert(kTileRows == 32 * WAVES, "the layout's tiles");
    static_assert(keys_of(HD) == 32 * KW, "the layout's chunks");
    hipError_t e;
    if (a.tiles > 0) {
        const dim3 grid(blocks_of((int64_t)a.tiles * a.H_kv * a.splits) + (local ? a.pads : 0)), block(64 * WAVES);   // some more for the rows of padding
        if (local) {
            if (a.edge) hipLaunchKernelGGL((train_dq_kernel<HD, WAVES, true, true>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((train_dq_kernel<HD, WAVES, false, true>), grid, block, 0, s, a);
        } else {
            if (a.edge) hipLaunchKernelGGL((train_dq_kernel<HD, WAVES, true, false>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((train_dq_kernel<HD, WAVES, false, false>), grid, block, 0, s, a);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.splits > 1) {
            hipLaunchKernelGGL((train_dq_join_kernel<HD>), dim3((unsigned)((int64_t)a.tiles * a.H_kv * kTileRows * HD * kJoiners / 1024)), dim3(256), 0, s, a);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    const dim3 grid(blocks_of((int64_t)a.chunks * a.H_kv * ((a.L_kv + keys_of(HD) - 1) / keys_of(HD))));
    const dim3 block(64 * KW);
    if (local) {
        if (a.edge) hipLaunchKernelGGL((train_dkv_kernel<HD, KW, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((train_dkv_kernel<HD, KW, false, true>), grid, block, 0, s, a);
    } else {
        if (a.edge) hipLaunchKernelGGL((train_dkv_kernel<HD, KW, true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((train_dkv_kernel<HD, KW, false, false>), grid, block, 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess || a.n_joins == 0) return e;
    hipLaunchKernelGGL((train_dkv_join_kernel<HD>), dim3((unsigned)((int64_t)a.n_joins * a.H_kv * ((a.L_kv + 15) / 16))), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_train_backward(const TrainArgs &a, const TrainLayout &w, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128, kRowWaves, 8>(a, w.local, s) : launch<64, kRowWaves, 4>(a, w.local, s);
}

}  // namespace ikbo
