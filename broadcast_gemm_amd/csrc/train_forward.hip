// train_forward.hip -- target attention that keeps its statistics (ikbo_attention_forward).
//
// The rows of one user and shared head (its candidates' queries, of all heads of the group) stand beside one another, 32
// to a result tile, and read the same K and V.  A block takes a tile of rows against a range of keys, 64 at a time: S^T =
// K Q^T, weights against a running maximum, O^T += V^T P^T.  K and V are staged in LDS (two buffers, loaded straight
// into it) and read there by all waves; V^T comes from transposed reads.  The maximum moves, and O is rescaled, only when
// it grows by more than 8 in base 2 (below: 151 us, 159 without this).  Weights are rounded to bf16 for the product (half a
// step of bf16 each, which the output's own rounding is too); their sums, and so lse, take them as they are, in float32.
// The scores of the next 64 keys stand beside the weights of these, so that the matrix cores work while exponentials are
// taken (162 -> 149 us); a second set of waves for every other stage of keys loses (192), as blocks of 8 waves do (180).
//
// Measured: 15 users, 1024 candidates of 64 queries, 4 heads of 128, 777 to 1024 tokens (121 GFLOP): 149 us, 810 TFLOP/s,
// where a library product of 8192^3 reaches 1378.  It is bound by what surrounds the products: six vector instructions for a
// matrix one, 32 exponentials a lane and stage; LDS reads meet no conflict.  26 users, 256 candidates of 33 queries, 8 heads
// of 64, dropout (11.4 GFLOP): 35 us; at head 64 the weights count double, and the generator's 28 wide products for 32
// tokens come to them.
//
// Few rows over long histories: the keys are cut into ranges, whose results a second launch joins (2 users of up to 32000
// tokens, 48 candidates, 53 MB: 22 us and 6.5 to join; 614 us uncut).
#include "train_device.h"

namespace ikbo {
namespace {

constexpr float kSlack = 8.0f;

template <int HD, int WAVES, bool DROP, bool LOCAL>
__global__ void __launch_bounds__(64 * WAVES, 2) train_fwd_kernel(TrainArgs a) {
    constexpr int TK = HD / 16, DT = HD / 32, STAGE = Rows<HD>::matrix(64), ROWS = 32 * WAVES;
    __shared__ __align__(16) char k_lds[2][STAGE], v_lds[2][STAGE];
    __shared__ int s_most[WAVES];
    if constexpr (LOCAL) {
        const int pad = (int)blockIdx.x - (int)gridDim.x + a.pads;
        if (pad >= 0) {   // the last blocks
            fill_padding(a, HD, false, pad);
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
    KeyLoads<HD, WAVES> keys;
    keys.init(a, u, hk, lane, wv);
    auto load_k = [&](int st) { keys.load_k(lds_address(k_lds[st & 1]), wv, key0 + 64 * st, len); };
    auto load_v = [&](int st) { keys.load_v(lds_address(v_lds[st & 1]), wv, key0 + 64 * st, len); };
    load_k(0);
    load_v(0);
    load_k(1);
    if constexpr (LOCAL) {
        local.list(a, s_local, u);
        if (a.splits > 1 && hk == 0 && split == 0 && row0 == 0)
            for (int i = tid; i * a.G * a.L_q < n_rows; i += 64 * WAVES) a.perm[t.first + i] = s_local.list[i];
    }
    auto place = [&](int r) {
        if constexpr (LOCAL) return place_of(a, s_local.list, hk, r);
        else return place_of(a, a.perm + t.first, hk, r);
    };
    // The lane's row.
    const int r = row0 + wv * 32 + j;
    const bool live = r < n_rows;
    int limit, most, least;
    uint32_t row, head;
    u32x4_t qf[TK];
    {
        const Place at = place(live ? r : 0);
        limit = live ? limit_of(a, at, len) : 0;
        row = (uint32_t)(at.cand * a.L_q + at.query);
        head = (uint32_t)at.head;
        const uint16_t *q = a.Q + at.cand * a.q_cand + at.head * a.q_head + at.query * a.q_query + 8 * g;
#pragma unroll
        for (int s = 0; s < TK; ++s) qf[s] = live ? *reinterpret_cast<const u32x4_t *>(q + 16 * s) : (u32x4_t){0, 0, 0, 0};
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
    if (lane == 0) s_most[wv] = most;
    __syncthreads();
    int end = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) end = max(end, s_most[w]);
    end = min(end, key0 + a.split_keys);
    // Stages of the block, and those in which a row of the wave sees a key.
    const int stages = __builtin_amdgcn_readfirstlane(max(0, (end - key0 + 63) >> 6)), mine = min(stages, max(0, (most - key0 + 63) >> 6));

    Random rnd;
    if constexpr (DROP) rnd.init(a.rng);
    f32x16_t o[DT];
    float m = neg_inf(), l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = (f32x16_t)(0.f);
    Reader<HD> rd;
    rd.init(lane);
    // S^T of keys 64 st + 32 h + 8 (i / 4) + 4 g + i % 4.
    auto scores = [&](int st, f32x16_t (&S)[2]) {
        const char *K = k_lds[st & 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            S[h] = (f32x16_t)(0.f);
#pragma unroll
            for (int s = 0; s < TK; ++s) S[h] = mfma32(rd.direct(K, h, s), qf[s], S[h]);
        }
    };
    // What the row does not see, and the running maximum.
    auto raise = [&](int st, f32x16_t (&S)[2]) {
        const int t0 = key0 + 64 * st;
        if (t0 + 64 > least) {
            asm volatile("");   // stays a branch: as selects its body would be paid by every stage
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (t0 + 32 * h + 8 * (i >> 2) + 4 * g + (i & 3) >= limit) S[h][i] = neg_inf();
        }
        float x = neg_inf();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) x = fmaxf(x, S[h][i]);
        const float top = max_halves(x) * a.scale_log2;
        if (__ballot(top > m + kSlack)) {
            const float now = fmaxf(m, top);
            const float by = now == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(m - now);
            m = now;
            l *= by;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= by;
        }
    };
    // Weights of stage st's scores, and O^T += V^T P^T.
    auto weigh = [&](int st, const f32x16_t (&S)[2]) {
        const char *V = v_lds[st & 1];
        u32x4_t pf[4];
        const float nm = m == neg_inf() ? 0.f : -m;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[h][i], a.scale_log2, nm));
                l += p[i];
            }
            if constexpr (DROP) {
                const u32x4_t w = rnd.weights(((key0 + 64 * st) >> 5) + h, g, row, head);
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = ((w[i >> 2] >> (8 * (i & 3))) & 255u) >= a.edge ? p[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) pf[2 * h + (i >> 3)][(i >> 1) & 3] = pack_bf16x2(p[i], p[i + 1]);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] = mfma32(rd.turned(V, s, d), pf[s], o[d]);
    };
    // At the top of turn st, K of stage st + 1 and V of st are in LDS and the scores of st in `now`; while the weights of
    // st are formed, the matrix cores take the scores of st + 1.
    f32x16_t even[2], odd[2];
    auto turn = [&](int st, f32x16_t (&now)[2], f32x16_t (&next)[2]) {
        if (st + 1 < stages) load_v(st + 1);
        if (st + 2 < stages) load_k(st + 2);
        if (st < mine) {
            scores(st + 1, next);   // of the last turn for nothing: a turn of its own without them would cost registers
            weigh(st, now);
            if (st + 1 < mine) raise(st + 1, next);
        }
        landed();
        __syncthreads();
    };
    landed();   // also where no stage is wanted: nothing may arrive after the block
    __syncthreads();
    if (stages > 0) {
        if (mine > 0) {
            scores(0, even);
            raise(0, even);
        }
        __syncthreads();   // K of stage 0 has been read
    }
    for (int st = 0; st < stages; st += 2) {
        turn(st, even, odd);
        if (st + 1 < stages) turn(st + 1, odd, even);
    }
    const float sum = sum_halves(l);
    if (!live) return;
    const Place at = place(r);   // again, rather than kept
    if (a.splits == 1) {
        const float by = sum > 0.f || sum != sum ? a.keep / sum : 0.f;   // a row that sees nothing is 0
        uint16_t *to = a.O + at.cand * a.o_cand + at.head * a.o_head + at.query * a.o_query + 8 * g;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int p = 0; p < 2; ++p) *reinterpret_cast<u32x4_t *>(to + 32 * d + 16 * p) = eight_rows(o[d], p, by);
        if (g == 0) a.lse[((int64_t)at.cand * a.H_q + at.head) * a.L_q + at.query] = m * kLn2 + logf(sum);
    } else {
        const int64_t part = (((int64_t)split * a.tiles + tile) * a.H_kv + hk) * ROWS + wv * 32 + j;
        float *to = a.part + part * HD + 4 * g;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4_t *>(to + 32 * d + 8 * q) = (f32x4_t){o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
        if (g == 0) a.ml[part] = make_float2(m, sum);
    }
}

// The parts of one row of O: kJoiners groups of HD / 4 lanes take every kJoiners-th each (170 parts: 6.4 us, 23 by one group).
// Bound by the chain of its loads.
template <int HD>
__global__ void __launch_bounds__(256) train_fwd_join_kernel(TrainArgs a) {
    constexpr int LANES = HD / 4, ROWS = 256 / LANES / kJoiners;
    __shared__ f32x4_t parts[kJoiners][ROWS][LANES];
    __shared__ float sums[kJoiners][ROWS];
    const int x = (int)threadIdx.x % LANES, row = (int)threadIdx.x / LANES % ROWS, part = (int)threadIdx.x / LANES / ROWS;
    const int64_t i = (int64_t)blockIdx.x * ROWS + row;
    const int in_tile = (int)(i % kTileRows), hk = (int)(i / kTileRows % a.H_kv), tile = (int)(i / kTileRows / a.H_kv);
    const TileEntry t = a.tile[min(tile, a.tiles - 1)];
    const int r = t.row + in_tile;
    const bool live = tile < a.tiles && t.user >= 0 && r < t.rows;
    const int64_t row0 = ((int64_t)tile * a.H_kv + hk) * kTileRows + in_tile, step = (int64_t)a.tiles * a.H_kv * kTileRows;
    float top = neg_inf(), sum = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        for (int s = x; s < a.splits; s += LANES) top = fmaxf(top, a.ml[row0 + s * step].x);
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll 4
        for (int s = part; s < a.splits; s += kJoiners) {
            const float2 ml = a.ml[row0 + s * step];
            const float w = ml.x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
            sum += w * ml.y;
            o += w * *reinterpret_cast<const f32x4_t *>(a.part + (row0 + s * step) * HD + 4 * x);
        }
    }
    parts[part][row][x] = o;
    if (x == 0) sums[part][row] = sum;
    __syncthreads();
    if (part > 0 || !live) return;
#pragma unroll
    for (int y = 1; y < kJoiners; ++y) {
        o += parts[y][row][x];
        sum += sums[y][row];
    }
    const float by = sum > 0.f || sum != sum ? a.keep / sum : 0.f;
    const Place p = place_of(a, a.perm + t.first, hk, r);
    *reinterpret_cast<u32x2_t *>(a.O + p.cand * a.o_cand + p.head * a.o_head + p.query * a.o_query + 4 * x) =
        (u32x2_t){pack_bf16x2(o[0] * by, o[1] * by), pack_bf16x2(o[2] * by, o[3] * by)};
    if (x == 0) a.lse[((int64_t)p.cand * a.H_q + p.head) * a.L_q + p.query] = top * kLn2 + logf(sum);
}

template <int HD, int WAVES>
hipError_t launch(const TrainArgs &a, bool local, hipStream_t s) {
    const dim3 grid(blocks_of((int64_t)a.tiles * a.H_kv * a.splits) + (local ? a.pads : 0)), block(64 * WAVES);   // some more for the rows of padding
    if (local) {
        if (a.edge) hipLaunchKernelGGL((train_fwd_kernel<HD, WAVES, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((train_fwd_kernel<HD, WAVES, false, true>), grid, block, 0, s, a);
    } else {
        if (a.edge) hipLaunchKernelGGL((train_fwd_kernel<HD, WAVES, true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((train_fwd_kernel<HD, WAVES, false, false>), grid, block, 0, s, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    static_assert(kTileRows == 32 * WAVES, "the layout's tiles");
    hipLaunchKernelGGL((train_fwd_join_kernel<HD>), dim3((unsigned)((int64_t)a.tiles * a.H_kv * kTileRows * HD * kJoiners / 1024)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_train_forward(const TrainArgs &a, const TrainLayout &w, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128, kRowWaves>(a, w.local, s) : launch<64, kRowWaves>(a, w.local, s);
}

}  // namespace ikbo
