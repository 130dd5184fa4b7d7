// train_prep.hip -- the first launch of attention's training calls: the candidates grouped by user, the work cut into
// blocks (TrainLayout), and the rows of padding filled in.
//
// Block 0 groups with a stable counting sort: a wave takes a run of candidates, 64 to a turn.  The lanes with the same
// key are found from ballots of the key's bits, whatever the map looks like.  Where queries have positions, the key is the
// user and a step of the candidate's position in the history, as many steps as LDS has counts for: rows that see about
// as many tokens then stand together, and their tiles end there (23 users, 8001 candidates: the grouping 10 -> 13 us,
// forward 80 -> 63, dQ 115 -> 89, dK and dV 122 -> 104).  The other blocks look for candidates whose map entry is no user,
// and write their O = 0 and lse = -inf, or dQ = 0.
//
// It is bound by latency: one block, and a dozen steps that wait for one another.  1024 candidates of 15 users 8 us, 8001 of
// 23 with positions 14.5, of which putting the tiles in order is 1.3.
#include <algorithm>

#include "train_device.h"

namespace ikbo {
namespace {

constexpr int kThreads = 1024;
constexpr int kMostSteps = 16, kBatch = 8;     // of the position; turns of a wave
constexpr int kOrders = 32;                   // of the tiles' work

// Exclusive prefix sums of v over the lanes of a wave; the totals in all.
template <int N>
__device__ __forceinline__ void scan_wave(int (&v)[N], int (&all)[N]) {
    const int lane = (int)threadIdx.x & 63;
    int own[N];
#pragma unroll
    for (int n = 0; n < N; ++n) own[n] = v[n];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int x = __shfl_up(v[n], d);
            if (lane >= d) v[n] += x;
        }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        all[n] = __shfl(v[n], 63);
        v[n] -= own[n];
    }
}

// The same over the block's threads; sh: 16 ints.
__device__ __forceinline__ int scan_block(int x, int &total, int *sh) {
    const int wv = (int)threadIdx.x >> 6;
    int v[1] = {x}, all[1];
    scan_wave(v, all);
    if ((threadIdx.x & 63) == 0) sh[wv] = all[0];
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; w += 4) {
        const int4 y = *reinterpret_cast<const int4 *>(sh + w);
        const int z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (w + i == wv) before = total;
            total += z[i];
        }
    }
    return v[0] + before;
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

__global__ void __launch_bounds__(kThreads) train_prep_kernel(TrainArgs a, int waves, int steps, int head_dim, int backward) {
    extern __shared__ int sh[];
    __shared__ __align__(16) int s_scan[kThreads / 64];
    __shared__ int s_orders[kOrders * kThreads / 64];
    __shared__ int s_total[5];   // tiles, chunks, slots, notes, joins
    if (blockIdx.x > 0) {
        fill_padding(a, head_dim, backward, (int)blockIdx.x - 1);
        return;
    }
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6, B = a.B_u, keys = B * steps;
    // Counts [waves][users * steps], then the users' offsets, prefix sums of tiles, chunks, slots and notes, and lengths.
    int *cnt = sh, *offs = sh + waves * keys, *t_at = offs + B + 1, *c_at = t_at + B + 1, *s_at = c_at + B + 1, *n_at = s_at + B + 1, *lens = n_at + B + 1;
    uint32_t err = 0;
    const int bits = 32 - __builtin_clz((unsigned)keys);
    const int seg = ((a.B_c + waves - 1) / waves + 63) / 64 * 64, lo = min(wv * seg, a.B_c), hi = wv < waves ? min(a.B_c, lo + seg) : lo;
    const uint64_t below = (1ull << lane) - 1;
    // kBatch turns of 64 candidates of the wave; what they read is under way together.  Of each candidate its key (-1: none)
    // and how many lanes before it, and in all, have the same.
    int key[kBatch], rank[kBatch], same_key[kBatch], pos[kBatch];
    auto fetch = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int b = b0 + 64 * i + lane;
            key[i] = b < hi ? a.map[b] : -1;
            pos[i] = steps > 1 && b < hi ? a.positions[(int64_t)b * a.L_q + a.L_q - 1] : 0;
            if (steps > 1 && a.L_q > 1 && b < hi) pos[i] = max(pos[i], a.positions[(int64_t)b * a.L_q]);
        }
    };
    fetch(lo);   // on its way before the lengths
    for (int u = tid; u < B; u += kThreads) {
        lens[u] = user_len(a, u);
        if (a.lens && a.lens[u] != lens[u]) err |= kTrainStLens;
    }
    for (int i = tid; i < waves * keys; i += kThreads) cnt[i] = 0;
    __syncthreads();
    auto find_keys = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b0 + 64 * i >= hi) continue;
            const int u = key[i];
            const bool valid = u >= 0 && u < B;
            if (!valid && u != -1) err = kTrainStMap;
            key[i] = valid ? u * steps : -1;
            if (steps > 1 && valid) {   // by the later of the first and the last query, far ones first
                const int len = lens[u];
                key[i] += steps - 1 - min(steps - 1, (int)((float)min(max(pos[i], 0), len) * (float)steps / (float)(len + 1)));
            }
            const uint64_t any = __ballot(valid);
            uint32_t same0 = (uint32_t)any, same1 = (uint32_t)(any >> 32);
            for (int k = 0; k < bits; ++k) {
                const uint32_t own = (uint32_t)((key[i] << (31 - k)) >> 31);   // the bit, everywhere
                const uint64_t m = __ballot(own != 0);
                same0 &= ~((uint32_t)m ^ own);
                same1 &= ~((uint32_t)(m >> 32) ^ own);
            }
            const uint64_t same = (uint64_t)same1 << 32 | same0;
            rank[i] = __popcll(same & below);
            same_key[i] = __popcll(same);
        }
    };
    // In the order of the candidates; of one batch the keys are still there the second time.
    const bool once = seg <= 64 * kBatch;
    auto walk = [&](bool again, auto each) __attribute__((always_inline)) {
        for (int b0 = lo; b0 < hi; b0 += 64 * kBatch) {
            if (!again || !once) {
                if (again || b0 > lo) fetch(b0);
                find_keys(b0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (b0 + 64 * i < hi && key[i] >= 0) each(b0 + 64 * i + lane, key[i], rank[i], same_key[i]);
        }
    };
    walk(false, [&](int, int k, int before, int all) {
        if (before == 0) cnt[wv * keys + k] += all;
    });
    __syncthreads();
    // Places in perm: those of each key, the waves one behind the other.
    const int each = (keys + kThreads - 1) / kThreads, k0 = min(keys, tid * each), k1 = min(keys, k0 + each);
    int at = 0, all;
    for (int k = k0; k < k1; ++k)
        for (int w = 0; w < waves; ++w) at += cnt[w * keys + k];
    at = scan_block(at, all, s_scan);
    for (int k = k0; k < k1; ++k) {
        if (k % steps == 0) offs[k / steps] = at;
        for (int w = 0; w < waves; ++w) {
            const int c = cnt[w * keys + k];
            cnt[w * keys + k] = at;
            at += c;
        }
    }
    if (tid == 0) offs[B] = all;
    __syncthreads();
    // The last wave, which has the fewest candidates, sums up the users; the others go on.  Chunks of a user's rows for dK
    // and dV: even ones, one at least (it writes the zeros of a user without candidates); the chunks of users with several
    // have places for partial results.
    const int GL = a.G * a.L_q;
    for (int u = tid; backward && u < B; u += kThreads) c_at[u] = max(1, ((offs[u + 1] - offs[u]) * GL + a.chunk_rows - 1) / a.chunk_rows);
    __syncthreads();
    if (wv == kThreads / 64 - 1) {
        const int per = (B + 63) / 64, u0 = min(B, lane * per), u1 = min(B, u0 + per);
        int c[5] = {0, 0, 0, 0, 0}, total[5];
        auto add = [&](int u) {
            const int rows = (offs[u + 1] - offs[u]) * GL, chunks = backward ? c_at[u] : 0;
            c[0] += (rows + kTileRows - 1) / kTileRows;
            c[1] += chunks;
            c[2] += chunks > 1 ? chunks : 0;
            c[3] += (rows + 63) / 64;
            c[4] += chunks > 1;
            return chunks;
        };
        for (int u = u0; u < u1; ++u) add(u);
        scan_wave(c, total);
        for (int u = u0; u < u1; ++u) {
            t_at[u] = c[0];
            s_at[u] = c[2];
            n_at[u] = c[3];
            const int first = c[1], slot = c[2], join = c[4], chunks = add(u);
            c_at[u] = first;
            if (chunks > 1) a.joins[join] = make_int4(u, lens[u], slot, chunks);
        }
        if (lane == 0) {
            t_at[B] = total[0];
            c_at[B] = total[1];
        }
        if (lane < 5) s_total[lane] = lane == 0 ? total[0] : lane == 1 ? total[1] : lane == 2 ? total[2] : lane == 3 ? total[3] : total[4];
    }
    walk(true, [&](int b, int k, int before, int all) {
        const int from = cnt[wv * keys + k];
        __builtin_amdgcn_wave_barrier();
        if (before == 0) cnt[wv * keys + k] = from + all;
        a.perm[from + before] = b;
    });
    __syncthreads();
    const auto tile = [&](int t) {
        if (t >= s_total[0]) return TileEntry{-1, 0, 0, 0, 0, 0, {0, 0}};
        const int u = find(t_at, B, t), row = (t - t_at[u]) * kTileRows;
        return TileEntry{u, row, offs[u], (offs[u + 1] - offs[u]) * GL, lens[u], n_at[u] + row / 64, {0, 0}};
    };
    if (a.tiles <= kThreads) {
        // Those that see most come first, so that no long block starts when the others end (59 users, 4096 candidates with positions:
        // forward 63 -> 47 us; 23 users, 8001 candidates: dQ 90 -> 68 us).  The order is a stable counting sort again; rows in the
        // order of their positions are taken to see evenly less and less.  More tiles than threads fill the card several times.
        const TileEntry x = tile(tid);
        const float sees = x.user < 0 ? 0.f : a.positions ? (float)x.len * (float)(x.rows - x.row) / (float)x.rows : (float)x.len;
        const int k = x.user < 0 ? kOrders - 1 : kOrders - 2 - min(kOrders - 2, (int)(sees * (float)(kOrders - 1) / (float)(a.L_kv + 1)));
        uint64_t same = ~0ull;
#pragma unroll
        for (int bit = 1; bit < kOrders; bit <<= 1) {
            const uint64_t m = __ballot(k & bit);
            same &= k & bit ? m : ~m;
        }
        if (tid < kOrders * kThreads / 64) s_orders[tid] = 0;
        __syncthreads();
        if ((same & below) == 0) s_orders[k * (kThreads / 64) + wv] = __popcll(same);
        __syncthreads();
        int total;
        const int n = tid < kOrders * kThreads / 64 ? s_orders[tid] : 0, before = scan_block(n, total, s_scan);
        if (tid < kOrders * kThreads / 64) s_orders[tid] = before;
        __syncthreads();
        const int to = s_orders[k * (kThreads / 64) + wv] + __popcll(same & below);
        if (to < a.tiles) a.tile[to] = x;
    } else {
        for (int t = tid; t < a.tiles; t += kThreads) a.tile[t] = tile(t);
    }
    for (int t = s_total[4] + tid; t < a.n_joins; t += kThreads) a.joins[t] = make_int4(0, 0, 0, 0);
    for (int t = tid; t < a.chunks; t += kThreads) {
        ChunkEntry x{-1, 0, 0, -1, 0, {0, 0, 0}};
        if (t < s_total[1]) {
            const int u = find(c_at, B, t), n = c_at[u + 1] - c_at[u], i = t - c_at[u];
            const int notes = ((offs[u + 1] - offs[u]) * GL + 63) / 64, some = (notes + n - 1) / n, from = min(notes, i * some);
            x = ChunkEntry{u, n_at[u] + from, min(notes, from + some) - from, n > 1 ? s_at[u] + i : -1, lens[u], {0, 0, 0}};
        }
        a.chunk[t] = x;
    }
    if (err) atomicOr(a.status, err);
}

}  // namespace

hipError_t launch_train_prep(const TrainArgs &a, bool backward, int head_dim, hipStream_t s) {
    // 156 KB of LDS hold the counts of 3 waves for the most users.
    constexpr int kInts = 39 * 1024;
    const int others_ints = 6 * (a.B_u + 1), room = kInts - others_ints;
    const int waves = std::min({kThreads / 64, std::max(1, (a.B_c + 255) / 256), room / a.B_u});
    const int steps = a.positions ? std::max(1, std::min(kMostSteps, room / (a.B_u * waves))) : 1;
    const int lds = 4 * (waves * a.B_u * steps + others_ints);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(train_prep_kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 4 * kInts);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(train_prep_kernel, dim3(1 + a.pads), dim3(kThreads), lds, s, a, waves, steps, head_dim, (int)backward);
    return hipGetLastError();
}

}  // namespace ikbo
