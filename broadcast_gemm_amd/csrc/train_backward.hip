// train_backward.hip -- the gradients of target attention (ikbo_attention_backward), probabilities recomputed.
//
// Two kernels, each with all it sums in registers, so that nothing is added up by atomics and no block waits for another:
//
// dQ: as the forward, a block takes a tile of rows against a range of keys: S^T = K Q^T, dP^T = V dO^T, P = exp(S - lse),
// dS = P (dP - D), dQ^T += K^T dS^T.  It first forms D = rowsum(dO O), which the other kernel reads.  For a row that
// sees no more than the first 64 keys D is the sum of P dP instead: with few keys the rounding of O shows in dP - D.
//
// dK and dV: a wave keeps 32 keys' K and V and their gradients in registers, and the block goes over a chunk of the
// user's rows, staged in LDS 64 at a time: S = Q K^T, dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS.  Rows stand in the
// results' rows here, so P and dS are the B operands as they stand.  The weights that stay are decided with the rows
// in the lanes, as in the other kernels (one generator call for 16 tokens of a row), and the bits turned round (Turn).  Chunks of one user are joined by a third launch, in their order.
//
// That is 7 products against the 5 that one pass needs; adding up dQ across key ranges instead would write and read 4
// bytes an element for every range.  P and dS are rounded to bf16 for their products; all sums are float32.
#include <algorithm>

#include "train_device.h"

namespace ikbo {
namespace {

template <int HD, int NT, int WAVES, bool DROP>
__global__ void __launch_bounds__(64 * WAVES, 1) train_dq_kernel(TrainArgs a) {
    constexpr int TK = HD / 16, DT = HD / 32, STAGE = Rows<HD>::matrix(64), ROWS = 32 * NT * WAVES;
    __shared__ __align__(16) char lds[2][2][STAGE];
    __shared__ int s_most[WAVES];
    const int n_tiles = a.count[0];
    const int unit = unit_of((int)blockIdx.x, n_tiles * a.H_kv * a.splits);
    if (unit < 0) return;   // the whole block: no barrier has run
    const int tile = unit % n_tiles, hk = unit / n_tiles % a.H_kv, split = unit / n_tiles / a.H_kv;
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5, j = lane & 31;
    const int u = __builtin_amdgcn_readfirstlane(a.tile[tile].x), row0 = __builtin_amdgcn_readfirstlane(a.tile[tile].y);
    const int first = a.off[u], n_rows = (a.off[u + 1] - first) * a.G * a.L_q, len = __builtin_amdgcn_readfirstlane(user_len(a, u));

    const int r0 = row0 + wv * 32 * NT;
    uint32_t row[NT], head[NT];
    int limit[NT], most = 0, least = len;
    bool live[NT];
    u32x4_t qf[TK][NT], gf[TK][NT];
    float shift[NT], D[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 32 * n + j;
        live[n] = r < n_rows;
        const Place at = place_of(a, first, hk, live[n] ? r : 0);
        limit[n] = live[n] ? limit_of(a, at, len) : 0;
        row[n] = (uint32_t)(at.cand * a.L_q + at.query);
        head[n] = (uint32_t)at.head;
        const bool sees = limit[n] > 0;   // other rows are not read: they have no gradient, whatever theirs is
        const uint16_t *q = a.Q + at.cand * a.q_cand + at.head * a.q_head + at.query * a.q_query + 8 * g;
        const uint16_t *dy = a.dO + at.cand * a.do_cand + at.head * a.do_head + at.query * a.do_query + 8 * g;
        const uint16_t *y = a.O + at.cand * a.o_cand + at.head * a.o_head + at.query * a.o_query + 8 * g;
        const int64_t stat = ((int64_t)at.cand * a.H_q + at.head) * a.L_q + at.query;
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < TK; ++s) {
            qf[s][n] = sees ? *reinterpret_cast<const u32x4_t *>(q + 16 * s) : (u32x4_t){0, 0, 0, 0};
            gf[s][n] = sees ? *reinterpret_cast<const u32x4_t *>(dy + 16 * s) : (u32x4_t){0, 0, 0, 0};
            const u32x4_t of = sees ? *reinterpret_cast<const u32x4_t *>(y + 16 * s) : (u32x4_t){0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum = __builtin_fmaf(__builtin_bit_cast(float, of[e] << 16), __builtin_bit_cast(float, gf[s][n][e] << 16), sum);
                sum = __builtin_fmaf(__builtin_bit_cast(float, of[e] & 0xFFFF0000u), __builtin_bit_cast(float, gf[s][n][e] & 0xFFFF0000u), sum);
            }
        }
        D[n] = sum_halves(sum);
        shift[n] = sees ? -a.lse[stat] * kLog2e : 0.f;
        most = max(most, limit[n]);
        if (live[n]) least = min(least, limit[n]);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        most = max(most, __shfl_xor(most, d));
        least = min(least, __shfl_xor(least, d));
    }
    most = __builtin_amdgcn_readfirstlane(most);
    least = __builtin_amdgcn_readfirstlane(least);
    if (lane == 0) s_most[wv] = most;
    __syncthreads();
    int end = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) end = max(end, s_most[w]);
    const int key0 = split * a.split_keys;
    end = min(end, key0 + a.split_keys);

    Random rnd;
    if constexpr (DROP) rnd.init(a.rng);
    f32x16_t dq[DT][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int d = 0; d < DT; ++d) dq[d][n] = (f32x16_t)(0.f);
    KeyLoads<HD, WAVES> keys;
    keys.init(a, u, hk, lane, wv);
    Reader<HD> rd;
    rd.init(lane);
    const uint32_t lds0 = lds_address(lds);
    const int stages = max(0, (end - key0 + 63) >> 6);
    if (stages > 0) keys.load(lds0, wv, key0, len);
    for (int st = 0; st < stages; ++st) {
        landed();
        __syncthreads();   // stage st is there, and its other buffer has been read
        if (st + 1 < stages) keys.load(lds0 + ((st + 1) & 1) * 2 * STAGE, wv, key0 + 64 * st + 64, len);
        const int t0 = key0 + 64 * st;
        if (t0 >= most) continue;   // none of the wave's rows sees these keys
        const char *K = lds[st & 1][0], *V = lds[st & 1][1];
        // P in S, and dP, of keys t0 + 32 h + 8 (i / 4) + 4 g + i % 4.
        f32x16_t S[NT], dP[NT];
        auto probabilities = [&](int h) {
#pragma unroll
            for (int n = 0; n < NT; ++n) S[n] = dP[n] = (f32x16_t)(0.f);
            u32x4_t kf[2], vf[2];
            kf[0] = rd.direct(K, h, 0);
            vf[0] = rd.direct(V, h, 0);
#pragma unroll
            for (int s = 0; s < TK; ++s) {
                if (s + 1 < TK) {
                    kf[(s + 1) & 1] = rd.direct(K, h, s + 1);
                    vf[(s + 1) & 1] = rd.direct(V, h, s + 1);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    S[n] = mfma32(kf[s & 1], qf[s][n], S[n]);
                    dP[n] = mfma32(vf[s & 1], gf[s][n], dP[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 16; ++i) S[n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[n][i], a.scale_log2, shift[n]));
                if constexpr (DROP) {
                    const u32x4_t w = rnd.weights((t0 >> 5) + h, g, row[n], head[n]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) dP[n][i] = ((w[i >> 2] >> (8 * (i & 3))) & 255u) >= a.edge ? dP[n][i] * a.keep : 0.f;
                }
            }
            if (t0 + 32 * h + 32 > least) {
                asm volatile("");   // stays a branch: as selects its body would be paid by every stage
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (t0 + 32 * h + 8 * (i >> 2) + 4 * g + (i & 3) >= limit[n]) S[n][i] = 0.f;
            }
        };
        if (t0 == 0 && least <= 64) {
            float sum[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) sum[n] = 0.f;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                probabilities(h);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[n] = __builtin_fmaf(S[n][i], dP[n][i], sum[n]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                sum[n] = sum_halves(sum[n]);
                D[n] = limit[n] <= 64 ? sum[n] : D[n];
            }
        }
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            probabilities(h);
            u32x4_t pf[2][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                    pf[i >> 3][n][(i >> 1) & 3] = pack_bf16x2(S[n][i] * (dP[n][i] - D[n]), S[n][i + 1] * (dP[n][i + 1] - D[n]));
                        u32x4_t kt[2];
            kt[0] = rd.turned(K, 2 * h, 0);
#pragma unroll
            for (int i = 0; i < 2 * DT; ++i) {
                if (i + 1 < 2 * DT) kt[(i + 1) & 1] = rd.turned(K, 2 * h + (i + 1) / DT, (i + 1) % DT);
#pragma unroll
                for (int n = 0; n < NT; ++n) dq[i % DT][n] = mfma32(kt[i & 1], pf[i / DT][n], dq[i % DT][n]);
                            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 32 * n + j;
        const Place to_row = place_of(a, first, hk, live[n] ? r : 0);   // again, rather than kept
        if (split == 0 && g == 0 && r < ((n_rows + 63) & ~63)) {
            RowNotes &x = a.notes[(int64_t)hk * a.n_notes + a.tile[tile].z + ((r - row0) >> 6)];
            const int i = r & 63;
            const bool sees = limit[n] > 0;
            x.q[i] = sees ? (const void *)(a.Q + to_row.cand * a.q_cand + to_row.head * a.q_head + to_row.query * a.q_query) : kZeroRow;
            x.dy[i] = sees ? (const void *)(a.dO + to_row.cand * a.do_cand + to_row.head * a.do_head + to_row.query * a.do_query) : kZeroRow;
            x.shift[i] = sees ? shift[n] : neg_inf();
            x.D[i] = D[n];
            x.limit[i] = limit[n];
            x.row[i] = to_row.cand * a.L_q + to_row.query;
            x.head[i] = to_row.head;
        }
        if (!live[n]) continue;
        if (a.splits == 1) {
            uint16_t *to = a.dQ + to_row.cand * a.dq_cand + to_row.head * a.dq_head + to_row.query * a.dq_query + 8 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int p = 0; p < 2; ++p) *reinterpret_cast<u32x4_t *>(to + 32 * d + 16 * p) = eight_rows(dq[d][n], p, a.scale);
        } else {
            float *to = a.part + ((((int64_t)split * a.tiles + tile) * a.H_kv + hk) * ROWS + wv * 32 * NT + 32 * n + j) * HD + 4 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4_t *>(to + 32 * d + 8 * q) = (f32x4_t){dq[d][n][4 * q], dq[d][n][4 * q + 1], dq[d][n][4 * q + 2], dq[d][n][4 * q + 3]};
        }
    }
}

// The parts of one row of dQ, by HD / 4 lanes, in the order of the keys.
template <int HD>
__global__ void __launch_bounds__(256) train_dq_join_kernel(TrainArgs a, int tile_rows) {
    constexpr int LANES = HD / 4;
    const int n_tiles = a.count[0], x = (int)threadIdx.x % LANES;
    const int64_t i = (int64_t)blockIdx.x * (256 / LANES) + (int)threadIdx.x / LANES, n = (int64_t)n_tiles * a.H_kv * tile_rows;
    if (i >= n) return;
    const int in_tile = (int)(i % tile_rows), hk = (int)(i / tile_rows % a.H_kv), tile = (int)(i / tile_rows / a.H_kv);
    const int u = a.tile[tile].x, r = a.tile[tile].y + in_tile, first = a.off[u];
    if (r >= (a.off[u + 1] - first) * a.G * a.L_q) return;
    const int64_t row0 = ((int64_t)tile * a.H_kv + hk) * tile_rows + in_tile, step = (int64_t)a.tiles * a.H_kv * tile_rows;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) o += *reinterpret_cast<const f32x4_t *>(a.part + (row0 + s * step) * HD + 4 * x);
    const Place p = place_of(a, first, hk, r);
    *reinterpret_cast<u32x2_t *>(a.dQ + p.cand * a.dq_cand + p.head * a.dq_head + p.query * a.dq_query + 4 * x) =
        (u32x2_t){pack_bf16x2(o[0] * a.scale, o[1] * a.scale), pack_bf16x2(o[2] * a.scale, o[3] * a.scale)};
}

template <int HD, int WAVES, bool DROP>
__global__ void __launch_bounds__(64 * WAVES, 1) train_dkv_kernel(TrainArgs a) {
    constexpr int TK = HD / 16, DT = HD / 32, STAGE = Rows<HD>::matrix(64), KEYS = 32 * WAVES, N = 64 * HD / 8 / (64 * WAVES);
    constexpr bool V_LDS = HD == 128;   // V stays in LDS: 32 registers less, which lets two waves stand on a SIMD
    __shared__ __align__(16) char lds[2][2][STAGE], v_lds[V_LDS ? Rows<HD>::matrix(KEYS) : 16];
    __shared__ __align__(16) RowNotes notes[3];
    const int n_chunks = a.count[1], ranges = (a.L_kv + KEYS - 1) / KEYS;
    const int unit = unit_of((int)blockIdx.x, n_chunks * a.H_kv * ranges);
    if (unit < 0) return;   // the whole block: no barrier has run
    const int range = unit % ranges, hk = unit / ranges % a.H_kv, c = unit / ranges / a.H_kv;   // neighbours share rows
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5, j = lane & 31;
    const int4 ch = a.chunk[c];
    const int u = __builtin_amdgcn_readfirstlane(ch.x), len = __builtin_amdgcn_readfirstlane(user_len(a, u));
    const int key0 = range * KEYS + wv * 32;

    const int token = Turn::token(j);   // of each 32 keys, the one in this lane
    Random rnd;
    Turn turn;
    if constexpr (DROP) {
        rnd.init(a.rng);
        turn.init(lane);
    }
    u32x4_t kf[TK], vf[V_LDS ? 1 : TK];
    f32x16_t dk[DT], dv[DT];
    {
        const int t = key0 + token;
        const uint16_t *k = a.K + u * a.k_user + hk * a.k_head + t * a.k_token + 8 * g;
        const uint16_t *v = a.V + u * a.v_user + hk * a.v_head + t * a.v_token + 8 * g;
#pragma unroll
        for (int s = 0; s < TK; ++s) {
            kf[s] = t < len ? *reinterpret_cast<const u32x4_t *>(k + 16 * s) : (u32x4_t){0, 0, 0, 0};
            if constexpr (!V_LDS) vf[s] = t < len ? *reinterpret_cast<const u32x4_t *>(v + 16 * s) : (u32x4_t){0, 0, 0, 0};
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) dk[d] = dv[d] = (f32x16_t)(0.f);
    }
    if constexpr (V_LDS) {   // each wave its own keys
        const uint16_t *v = a.V + u * a.v_user + hk * a.v_head;
#pragma unroll
        for (int i = 0; i < 32 * HD / 8 / 64; ++i) {
            const int p = i * 64 + lane, row = p / Rows<HD>::CHUNKS, chunk = ((p % Rows<HD>::CHUNKS) ^ Rows<HD>::number(row)) * 16;
            const int t = key0 + Turn::token(row);
            load_to_lds(t < len ? reinterpret_cast<const char *>(v + t * a.v_token) + chunk : reinterpret_cast<const char *>(kZeroRow) + chunk,
                        lds_address(v_lds) + Rows<HD>::matrix(32) * wv + i * Rows<HD>::GROUP);
        }
    }
    Reader<HD> rd;
    rd.init(lane);
    const uint32_t lds0 = lds_address(lds);
    const int stages = range * KEYS < len ? __builtin_amdgcn_readfirstlane(ch.z) : 0;   // keys behind the history: zeros
    const char *from_notes = reinterpret_cast<const char *>(a.notes + (int64_t)hk * a.n_notes + ch.y) + 16 * lane;
    auto load_notes = [&](int st) {
#pragma unroll
        for (int i = 0; i < 3; ++i) load_to_lds(from_notes + st * 3072 + 1024 * i, lds_address(&notes[st % 3]) + 1024 * i);
    };
    auto load = [&](int st) {
        const RowNotes &x = notes[st % 3];
        const uint32_t to = lds0 + (st & 1) * 2 * STAGE;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = (i * WAVES + wv) * 64 + lane, row = p / Rows<HD>::CHUNKS;
            const int chunk = ((p % Rows<HD>::CHUNKS) ^ Rows<HD>::number(row)) * 16;
            load_to_lds(static_cast<const char *>(x.q[row]) + chunk, to + (i * WAVES + wv) * Rows<HD>::GROUP);
            load_to_lds(static_cast<const char *>(x.dy[row]) + chunk, to + STAGE + (i * WAVES + wv) * Rows<HD>::GROUP);
        }
    };
    if (stages > 0) {
        if (wv == 0) load_notes(0);
        if (wv == 0 && stages > 1) load_notes(1);
        landed();
        __syncthreads();
        load(0);
    }
    for (int st = 0; st < stages; ++st) {
        landed();
        __syncthreads();   // stage st and the notes of the next are there, and the other buffer has been read
        if (st + 1 < stages) load(st + 1);
        if (wv == 0 && st + 2 < stages) load_notes(st + 2);
        const RowNotes &x = notes[st % 3];
        const int limit = x.limit[lane];
        if (!__ballot(limit > key0)) continue;   // no row sees the wave's keys
        const bool partly = __ballot(limit < key0 + 32) != 0;
        const char *Q = lds[st & 1][0], *Y = lds[st & 1][1];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            // Operands are read one step ahead of their products; the fences keep the compiler from reading further ahead,
            // for which it would spill: a spilled register's load would wait for the next stage's.
            f32x16_t S, dP;
            S = dP = (f32x16_t)(0.f);
            u32x4_t qf[2], yf[2], vl[2];
            auto operands = [&](int s) {
                qf[s & 1] = rd.direct(Q, h, s);
                yf[s & 1] = rd.direct(Y, h, s);
                if constexpr (V_LDS) vl[s & 1] = rd.direct(v_lds + Rows<HD>::matrix(32) * wv, 0, s);
            };
            operands(0);
#pragma unroll
            for (int s = 0; s < TK; ++s) {
                if (s + 1 < TK) operands(s + 1);
                S = mfma32(qf[s & 1], kf[s], S);
                dP = mfma32(yf[s & 1], V_LDS ? vl[s & 1] : vf[V_LDS ? 0 : s], dP);
                fence<HD == 128>();
            }
            uint32_t stays = 0;
            if constexpr (DROP) stays = turn.rows(rnd.weights(key0 >> 5, g, (uint32_t)x.row[32 * h + j], (uint32_t)x.head[32 * h + j]), a.edge) >> (4 * g);
            u32x4_t pf[2], sf[2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // rows 8 q + 4 g + e
                const f32x4_t shift = *reinterpret_cast<const f32x4_t *>(x.shift + 32 * h + 8 * q + 4 * g);
                const f32x4_t D = *reinterpret_cast<const f32x4_t *>(x.D + 32 * h + 8 * q + 4 * g);
                float p[4], ds[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[4 * q + e], a.scale_log2, shift[e]));
                if (partly) {
                    asm volatile("");
                    const u32x4_t limits = *reinterpret_cast<const u32x4_t *>(x.limit + 32 * h + 8 * q + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = key0 + token < (int)limits[e] ? p[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float dp = dP[4 * q + e];
                    const bool stay = !DROP || (stays >> (8 * q + e) & 1);
                    if constexpr (DROP) dp = stay ? dp * a.keep : 0.f;
                    ds[e] = p[e] * (dp - D[e]);
                    p[e] = stay ? p[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pf[q >> 1][2 * (q & 1) + e] = pack_bf16x2(p[2 * e], p[2 * e + 1]);
                    sf[q >> 1][2 * (q & 1) + e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
                }
                fence<HD == 128>();
            }
            u32x4_t yt[2], qt[2];
            auto turned = [&](int i) {
                yt[i & 1] = rd.turned(Y, 2 * h + i / DT, i % DT);
                qt[i & 1] = rd.turned(Q, 2 * h + i / DT, i % DT);
            };
            turned(0);
#pragma unroll
            for (int i = 0; i < 2 * DT; ++i) {
                if (i + 1 < 2 * DT) turned(i + 1);
                dv[i % DT] = mfma32(yt[i & 1], pf[i / DT], dv[i % DT]);
                dk[i % DT] = mfma32(qt[i & 1], sf[i / DT], dk[i % DT]);
                fence<HD == 128>();
            }
        }
    }
    const int t = key0 + token;
    if (t < a.L_kv) {
        if (ch.w < 0) {
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
            const int64_t row = ((int64_t)ch.w * a.H_kv + hk) * a.L_kv + t;
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

// One key's dK and dV from the chunks of its user, by HD / 4 lanes, in the order of the chunks.
template <int HD>
__global__ void __launch_bounds__(256) train_dkv_join_kernel(TrainArgs a) {
    constexpr int LANES = HD / 4;
    const int x = (int)threadIdx.x % LANES;
    const int64_t heads = (int64_t)a.L_kv * a.H_kv;
    for (int64_t i = (int64_t)blockIdx.x * (256 / LANES) + (int)threadIdx.x / LANES; i < heads * a.B_u; i += (int64_t)gridDim.x * (256 / LANES)) {
        const int u = (int)(i / heads), hk = (int)(i / a.L_kv % a.H_kv), t = (int)(i % a.L_kv);
        const int2 mine = a.user_chunk[u];
        if (mine.y == 0) continue;   // written by its one chunk
        f32x4_t k = {0.f, 0.f, 0.f, 0.f}, v = {0.f, 0.f, 0.f, 0.f};
        if (t < user_len(a, u)) {
    #pragma unroll 4
            for (int c = 0; c < mine.y; ++c) {
                const int64_t row = ((int64_t)(mine.x + c) * a.H_kv + hk) * a.L_kv + t;
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

template <int HD, int NT, int WAVES, int KW>
hipError_t launch(const TrainArgs &a, hipStream_t s) {
    constexpr int ROWS = 32 * NT * WAVES, KEYS = 32 * KW, EACH = 1024 / HD;
    static_assert(KEYS == kKeys, "the layout's chunks");
    hipError_t e;
    if (a.tiles > 0) {
        const dim3 grid((unsigned)(((int64_t)a.tiles * a.H_kv * a.splits + 7) / 8 * 8));
        if (a.edge) hipLaunchKernelGGL((train_dq_kernel<HD, NT, WAVES, true>), grid, dim3(64 * WAVES), 0, s, a);
        else hipLaunchKernelGGL((train_dq_kernel<HD, NT, WAVES, false>), grid, dim3(64 * WAVES), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.splits > 1) {
            hipLaunchKernelGGL((train_dq_join_kernel<HD>), dim3((unsigned)(((int64_t)a.tiles * a.H_kv * ROWS + EACH - 1) / EACH)), dim3(256), 0, s, a, ROWS);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    const dim3 grid((unsigned)(((int64_t)a.chunks * a.H_kv * ((a.L_kv + KEYS - 1) / KEYS) + 7) / 8 * 8));
    if (a.edge) hipLaunchKernelGGL((train_dkv_kernel<HD, KW, true>), grid, dim3(64 * KW), 0, s, a);
    else hipLaunchKernelGGL((train_dkv_kernel<HD, KW, false>), grid, dim3(64 * KW), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess || a.slots == 0) return e;
    hipLaunchKernelGGL((train_dkv_join_kernel<HD>), dim3((unsigned)std::min<int64_t>(((int64_t)a.B_u * a.H_kv * a.L_kv + EACH - 1) / EACH, 1 << 16)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_train_backward(const TrainArgs &a, const TrainLayout &, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128, 1, 8, 8>(a, s) : launch<64, 1, 8, 8>(a, s);
}

}  // namespace ikbo
