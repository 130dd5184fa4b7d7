// train_forward.hip -- target attention that keeps its statistics (ikbo_attention_forward).
//
// The rows of one user and shared head (its candidates' queries, of all heads of the group) stand beside one another, 32
// to a result tile, and read the same K and V.  A block takes a tile of rows against a range of keys, 64 at a time: S^T =
// K Q^T, weights against a running maximum, O^T += V^T P^T.  K and V are staged in LDS (two buffers, loaded straight
// into it) and read there by all waves; V^T comes from transposed reads.  The maximum moves, and O is rescaled, only when
// it grows by more than 8 in base 2.  Weights are rounded to bf16 for the product (half a step of bf16 each, which the
// output's own rounding is too); their sums, and so lse, take them as they are, in float32.
//
// Few rows over long histories: the keys are cut into ranges, whose results a second launch joins.
#include "train_device.h"

namespace ikbo {
namespace {

constexpr float kSlack = 8.0f;

template <int HD, int NT, int WAVES, bool DROP>
__global__ void __launch_bounds__(64 * WAVES, 1) train_fwd_kernel(TrainArgs a) {
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

    // The wave's rows: 32 n + j.
    const int r0 = row0 + wv * 32 * NT;
    uint32_t row[NT], head[NT];
    int limit[NT], most = 0, least = len;
    bool live[NT];
    u32x4_t qf[TK][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = r0 + 32 * n + j;
        live[n] = r < n_rows;
        const Place at = place_of(a, first, hk, live[n] ? r : 0);
        limit[n] = live[n] ? limit_of(a, at, len) : 0;
        row[n] = (uint32_t)(at.cand * a.L_q + at.query);
        head[n] = (uint32_t)at.head;
        const uint16_t *q = a.Q + at.cand * a.q_cand + at.head * a.q_head + at.query * a.q_query + 8 * g;
#pragma unroll
        for (int s = 0; s < TK; ++s) qf[s][n] = live[n] ? *reinterpret_cast<const u32x4_t *>(q + 16 * s) : (u32x4_t){0, 0, 0, 0};
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
    f32x16_t o[DT][NT];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = neg_inf();
        l[n] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d][n] = (f32x16_t)(0.f);
    }
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
        f32x16_t S[2][NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int n = 0; n < NT; ++n) S[h][n] = (f32x16_t)(0.f);
#pragma unroll
            for (int s = 0; s < TK; ++s) {
                const u32x4_t kf = rd.direct(K, h, s);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[h][n] = mfma32(kf, qf[s][n], S[h][n]);
            }
        }
        if (t0 + 64 > least) {
            asm volatile("");   // stays a branch: as selects its body would be paid by every stage
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (t0 + 32 * h + 8 * (i >> 2) + 4 * g + (i & 3) >= limit[n]) S[h][n][i] = neg_inf();
        }
        bool grow = false;
        float top[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x = neg_inf();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) x = fmaxf(x, S[h][n][i]);
            top[n] = max_halves(x) * a.scale_log2;
            grow = grow || top[n] > m[n] + kSlack;
        }
        if (__ballot(grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float now = fmaxf(m[n], top[n]);
                const float by = now == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(m[n] - now);
                m[n] = now;
                l[n] *= by;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d][n] *= by;
            }
        }
        u32x4_t pf[4][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float nm = m[n] == neg_inf() ? 0.f : -m[n];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[h][n][i], a.scale_log2, nm));
                    l[n] += p[i];
                }
                if constexpr (DROP) {
                    const u32x4_t w = rnd.weights((t0 >> 5) + h, g, row[n], head[n]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[i] = ((w[i >> 2] >> (8 * (i & 3))) & 255u) >= a.edge ? p[i] : 0.f;
                }
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    pf[2 * h + s][n] = (u32x4_t){pack_bf16x2(p[8 * s], p[8 * s + 1]), pack_bf16x2(p[8 * s + 2], p[8 * s + 3]),
                                                 pack_bf16x2(p[8 * s + 4], p[8 * s + 5]), pack_bf16x2(p[8 * s + 6], p[8 * s + 7])};
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4_t vf = rd.turned(V, s, d);
#pragma unroll
                for (int n = 0; n < NT; ++n) o[d][n] = mfma32(vf, pf[s][n], o[d][n]);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float sum = sum_halves(l[n]);
        if (!live[n]) continue;
        const Place to_row = place_of(a, first, hk, r0 + 32 * n + j);   // again, rather than kept
        if (a.splits == 1) {
            const float by = sum > 0.f || sum != sum ? a.keep / sum : 0.f;   // a row that sees nothing is 0
            uint16_t *to = a.O + to_row.cand * a.o_cand + to_row.head * a.o_head + to_row.query * a.o_query + 8 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int p = 0; p < 2; ++p) *reinterpret_cast<u32x4_t *>(to + 32 * d + 16 * p) = eight_rows(o[d][n], p, by);
            if (g == 0) a.lse[((int64_t)to_row.cand * a.H_q + to_row.head) * a.L_q + to_row.query] = m[n] * kLn2 + logf(sum);
        } else {
            const int64_t at = (((int64_t)split * a.tiles + tile) * a.H_kv + hk) * ROWS + wv * 32 * NT + 32 * n + j;
            float *to = a.part + at * HD + 4 * g;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<f32x4_t *>(to + 32 * d + 8 * q) = (f32x4_t){o[d][n][4 * q], o[d][n][4 * q + 1], o[d][n][4 * q + 2], o[d][n][4 * q + 3]};
            if (g == 0) a.ml[at] = make_float2(m[n], sum);
        }
    }
}

// The parts of one row of O, by HD / 4 lanes.
template <int HD>
__global__ void __launch_bounds__(256) train_fwd_join_kernel(TrainArgs a, int tile_rows) {
    constexpr int LANES = HD / 4;
    const int n_tiles = a.count[0], x = (int)threadIdx.x % LANES;
    const int64_t i = (int64_t)blockIdx.x * (256 / LANES) + (int)threadIdx.x / LANES, n = (int64_t)n_tiles * a.H_kv * tile_rows;
    if (i >= n) return;
    const int in_tile = (int)(i % tile_rows), hk = (int)(i / tile_rows % a.H_kv), tile = (int)(i / tile_rows / a.H_kv);
    const int u = a.tile[tile].x, r = a.tile[tile].y + in_tile, first = a.off[u];
    if (r >= (a.off[u + 1] - first) * a.G * a.L_q) return;
    const int64_t row0 = ((int64_t)tile * a.H_kv + hk) * tile_rows + in_tile, step = (int64_t)a.tiles * a.H_kv * tile_rows;
    float top = neg_inf(), sum = 0.f;
    for (int s = x; s < a.splits; s += LANES) top = fmaxf(top, a.ml[row0 + s * step].x);
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = a.ml[row0 + s * step];
        const float w = ml.x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
        sum += w * ml.y;
        o += w * *reinterpret_cast<const f32x4_t *>(a.part + (row0 + s * step) * HD + 4 * x);
    }
    const float by = sum > 0.f || sum != sum ? a.keep / sum : 0.f;
    const Place p = place_of(a, first, hk, r);
    *reinterpret_cast<u32x2_t *>(a.O + p.cand * a.o_cand + p.head * a.o_head + p.query * a.o_query + 4 * x) =
        (u32x2_t){pack_bf16x2(o[0] * by, o[1] * by), pack_bf16x2(o[2] * by, o[3] * by)};
    if (x == 0) a.lse[((int64_t)p.cand * a.H_q + p.head) * a.L_q + p.query] = top * kLn2 + logf(sum);
}

template <int HD, int NT, int WAVES>
hipError_t launch(const TrainArgs &a, hipStream_t s) {
    const int64_t units = (int64_t)a.tiles * a.H_kv * a.splits;
    const dim3 grid((unsigned)((units + 7) / 8 * 8));
    if (a.edge) hipLaunchKernelGGL((train_fwd_kernel<HD, NT, WAVES, true>), grid, dim3(64 * WAVES), 0, s, a);
    else hipLaunchKernelGGL((train_fwd_kernel<HD, NT, WAVES, false>), grid, dim3(64 * WAVES), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    constexpr int ROWS = 32 * NT * WAVES, EACH = 1024 / HD;
    hipLaunchKernelGGL((train_fwd_join_kernel<HD>), dim3((unsigned)(((int64_t)a.tiles * a.H_kv * ROWS + EACH - 1) / EACH)), dim3(256), 0, s, a, ROWS);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_train_forward(const TrainArgs &a, const TrainLayout &, int head_dim, hipStream_t s) {
    return head_dim == 128 ? launch<128, 1, 8>(a, s) : launch<64, 1, 8>(a, s);
}

}  // namespace ikbo
