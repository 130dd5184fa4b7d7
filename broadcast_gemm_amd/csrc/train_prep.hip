// train_prep.hip -- the first launch of attention's training calls: the candidates grouped by user, the work cut into
// blocks (TrainLayout), and the rows of padding filled in.
//
// Block 0 groups with a stable counting sort: a wave takes a run of candidates, 64 at a time.  The lanes with the same
// user are found from ballots of the user's bits, 12 at most, whatever the map looks like.  The other blocks look for
// candidates whose map entry is no user, and write their O = 0 and lse = -inf, or dQ = 0.
#include <algorithm>

#include "train_device.h"

namespace ikbo {
namespace {

constexpr int kThreads = 1024, kMaxUsers = IKBO_KV_MAX_USERS;
constexpr int kPer = kMaxUsers / kThreads;     // users per thread, at most

// Ints of LDS besides the counts per wave: the users' offsets, and prefix sums of tiles, chunks, slots and notes.
__host__ __device__ inline int prep_ints(int B_u, int waves) { return waves * B_u + 5 * (B_u + 1); }

// Exclusive prefix sums over the block's threads of v[0..N); totals in all.  sh: 16 N ints.
template <int N>
__device__ __forceinline__ void scan(int (&v)[N], int (&all)[N], int *sh) {
    const int lane = (int)threadIdx.x & 63, wv = (int)threadIdx.x >> 6;
    int own[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        own[n] = v[n];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(v[n], d);
            if (lane >= d) v[n] += x;
        }
        if (lane == 63) sh[16 * n + wv] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        int before = 0;
        all[n] = 0;
        for (int w = 0; w < 16; ++w) {
            if (w == wv) before = all[n];
            all[n] += sh[16 * n + w];
        }
        v[n] += before - own[n];
    }
    __syncthreads();
}

// The last i with at[i] <= x.
__device__ __forceinline__ int find(const int *at, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ void fill_padding(const TrainArgs &a, int head_dim, bool backward) {
    const int n = a.H_q * a.L_q, lane = (int)threadIdx.x & 63;
    const int w = ((int)blockIdx.x - 1) * (kThreads / 64) + ((int)threadIdx.x >> 6), waves = ((int)gridDim.x - 1) * (kThreads / 64);
    for (int b0 = w * 64; b0 < a.B_c; b0 += waves * 64) {
        const int u = b0 + lane < a.B_c ? a.map[b0 + lane] : 0;
        uint64_t none = __ballot(u < 0 || u >= a.B_u);
        while (none) {
            const int b = b0 + __ffsll((unsigned long long)none) - 1;
            none &= none - 1;
            uint16_t *to = backward ? a.dQ + b * a.dq_cand : a.O + b * a.o_cand;
            const int64_t head = backward ? a.dq_head : a.o_head, query = backward ? a.dq_query : a.o_query;
            for (int i = lane; i < n * (head_dim / 8); i += 64) {
                const int r = i / (head_dim / 8), h = r / a.L_q;
                *reinterpret_cast<u32x4_t *>(to + h * head + (r - h * a.L_q) * query + 8 * (i % (head_dim / 8))) = (u32x4_t){0, 0, 0, 0};
            }
            if (!backward)
                for (int i = lane; i < n; i += 64) a.lse[(int64_t)b * n + i] = neg_inf();
        }
    }
}

__global__ void __launch_bounds__(kThreads) train_prep_kernel(TrainArgs a, int waves, int tile_rows, int head_dim, int backward) {
    extern __shared__ int sh[];
    __shared__ int s_scan[64];   // 16 waves, 4 sums
    if (blockIdx.x > 0) {
        fill_padding(a, head_dim, backward);
        return;
    }
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6, B = a.B_u;
    int *cnt = sh, *offs = sh + waves * B, *t_at = offs + B + 1, *c_at = t_at + B + 1, *s_at = c_at + B + 1, *n_at = s_at + B + 1;
    uint32_t err = 0;
    for (int i = tid; i < waves * B; i += kThreads) cnt[i] = 0;
    __syncthreads();
    const int bits = 32 - __builtin_clz((unsigned)B);
    const int seg = ((a.B_c + waves - 1) / waves + 63) / 64 * 64, lo = min(wv * seg, a.B_c), hi = min(a.B_c, lo + seg);
    auto walk = [&](auto each) {
        if (wv < waves)
            for (int b0 = lo, next = lo + lane < hi ? a.map[lo + lane] : -1; b0 < hi; b0 += 64) {
                const int b = b0 + lane, u = next;
                next = b + 64 < hi ? a.map[b + 64] : -1;
                const bool valid = u >= 0 && u < B;
                if (!valid && u != -1) err = kTrainStMap;
                uint64_t same = __ballot(valid);
                for (int i = 0; i < bits; ++i) {
                    const uint64_t m = __ballot((u >> i) & 1);
                    same &= (u >> i) & 1 ? m : ~m;
                }
                if (valid) each(b, u, same);
            }
    };
    const uint64_t below = (1ull << lane) - 1;
    walk([&](int, int u, uint64_t same) {
        if ((same & below) == 0) cnt[wv * B + u] += __popcll(same);
    });
    __syncthreads();
    const int per = (B + kThreads - 1) / kThreads;
    int n_u[kPer], v[1] = {0}, all[1];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        n_u[e] = 0;
        if (e < per && u < B)
            for (int w = 0; w < waves; ++w) {
                const int c = cnt[w * B + u];
                cnt[w * B + u] = n_u[e];
                n_u[e] += c;
            }
        v[0] += n_u[e];
    }
    scan(v, all, s_scan);
    // Chunks of a user's rows for dK and dV: even ones, one at least (it writes the zeros of a user without candidates);
    // the chunks of users with several have places for partial results.
    int c[4] = {0, 0, 0, 0}, n_t[kPer], n_c[kPer], at = v[0];
    const int GL = a.G * a.L_q;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        n_t[e] = n_c[e] = 0;
        if (e < per && u < B) {
            offs[u] = at;
            at += n_u[e];
            const int rows = n_u[e] * GL;
            n_t[e] = (rows + tile_rows - 1) / tile_rows;
            n_c[e] = backward ? max(1, (rows + a.chunk_rows - 1) / a.chunk_rows) : 0;
            c[0] += n_t[e];
            c[1] += n_c[e];
            c[2] += n_c[e] > 1 ? n_c[e] : 0;
            c[3] += (rows + 63) / 64;
            if (a.lens && (a.lens[u] < 0 || a.lens[u] > a.L_kv)) err |= kTrainStLens;
        }
    }
    int total[4];
    scan(c, total, s_scan);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        if (e < per && u < B) {
            t_at[u] = c[0];
            c_at[u] = c[1];
            s_at[u] = c[2];
            n_at[u] = c[3];
            if (backward) a.user_chunk[u] = make_int2(c[2], n_c[e] > 1 ? n_c[e] : 0);
            c[0] += n_t[e];
            c[1] += n_c[e];
            c[2] += n_c[e] > 1 ? n_c[e] : 0;
            c[3] += (n_u[e] * GL + 63) / 64;
        }
    }
    if (tid == 0) {
        offs[B] = all[0];
        t_at[B] = total[0];
        c_at[B] = total[1];
        a.count[0] = total[0];
        a.count[1] = total[1];
    }
    __syncthreads();
    walk([&](int b, int u, uint64_t same) {
        const int first = cnt[wv * B + u];
        __builtin_amdgcn_wave_barrier();
        if ((same & below) == 0) cnt[wv * B + u] = first + __popcll(same);
        a.perm[offs[u] + first + __popcll(same & below)] = b;
    });
    for (int u = tid; u <= B; u += kThreads) a.off[u] = offs[u];
    for (int t = tid; t < total[0]; t += kThreads) {
        const int u = find(t_at, B, t);
        const int r = (t - t_at[u]) * tile_rows;
        a.tile[t] = make_int4(u, r, n_at[u] + r / 64, 0);
    }
    for (int t = tid; t < total[1]; t += kThreads) {
        const int u = find(c_at, B, t), n = c_at[u + 1] - c_at[u], i = t - c_at[u];
        const int blocks = ((offs[u + 1] - offs[u]) * GL + 63) / 64, each = (blocks + n - 1) / n, from = min(blocks, i * each);
        a.chunk[t] = make_int4(u, n_at[u] + from, min(blocks, from + each) - from, n > 1 ? s_at[u] + i : -1);
    }
    if (err) atomicOr(a.status, err);
}

}  // namespace

hipError_t launch_train_prep(const TrainArgs &a, int tile_rows, bool backward, int head_dim, hipStream_t s) {
    // 160 KB of LDS hold the counts of 8 waves for the most users.
    constexpr int kInts = 39 * 1024;
    const int need = std::max(1, (a.B_c + 255) / 256);
    const int waves = std::min({kThreads / 64, need, (kInts - prep_ints(a.B_u, 0)) / a.B_u});
    const int lds = 4 * prep_ints(a.B_u, waves);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(train_prep_kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 4 * kInts);
    if (e != hipSuccess) return e;
    const int others = std::min(64, (a.B_c + 1023) / 1024);
    hipLaunchKernelGGL(train_prep_kernel, dim3(1 + others), dim3(kThreads), lds, s, a, waves, tile_rows, head_dim, (int)backward);
    return hipGetLastError();
}

}  // namespace ikbo
