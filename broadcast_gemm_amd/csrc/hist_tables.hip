// hist_tables.hip -- page tables, slots, positions and rows of one step (ikbo_kv_tables).
//
// With the exclusive prefix sums over the requests of new tokens (starts), pages taken and pages
// returned, every output has a closed form: token row t belongs to the request i with
// starts[i] <= t < starts[i+1]; page p of the taken ones is ring[head + p] and belongs to the
// request whose range of the second sum holds p; likewise the returned ones.  So no block needs
// another's result: each block forms the three sums itself (at most 4096 requests, a few loads
// and one block-wide scan) and then takes its share of the rows and pages, found by binary search
// in LDS.  One launch, no waiting between blocks.
//
// In-place lengths and ring state may only change once every block has read them: a block counts
// itself in state[2] when it is done, and the last one writes lens_out and state_out and sets the
// count back to 0.  The ring's popped and pushed places are disjoint (their sum is at most the
// ring), and so are the table entries read (the page a request's next token falls into) and
// written (the ones behind it): those are updated where they are.
#include "hist_internal.h"

#include <algorithm>

namespace ikbo {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = IKBO_KV_MAX_USERS / kThreads;   // requests per thread

struct Sums {
    long long tok, take, give;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) { return {a.tok + b.tok, a.take + b.take, a.give + b.give}; }

// Largest i in [0, n) with base[i] <= x (base ascending, base[0] = 0 <= x).
__device__ __forceinline__ int owner_of(const int *base, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) kv_tables_kernel(ikbo_kv_tables_args a) {
    extern __shared__ int sh[];
    const int B = a.B_u, P = a.page_size, N = a.num_pages;
    int *s_tok = sh, *s_take = sh + B + 1, *s_give = sh + 2 * (B + 1);
    __shared__ Sums wsum[kThreads / 64];
    __shared__ uint32_t s_err;
    __shared__ int s_last;
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const long long head = a.state[0], nfree = a.state[1];
    if (tid == 0) s_err = (head < 0 || head >= N || nfree < 0 || nfree > N) ? kStPage : 0u;
    __syncthreads();

    // Each thread sums its consecutive requests, then a scan over the threads.
    const int per = (B + kThreads - 1) / kThreads;
    Sums mine{0, 0, 0}, part[kPer];
    uint32_t err = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = tid * per + e;
        Sums v{0, 0, 0};
        if (e < per && i < B) {
            const long long len = a.lens[i], c = a.counts[i], most = (long long)a.max_pages * P;
            if (len < 0 || len > most || c < -1) err |= kStPage;
            else if (c >= 0 && len + c > most) err |= kStNoPages;
            else {
                const int have = (int)((len + P - 1) / P);
                if (c < 0) v.give = have;
                else { v.tok = c; v.take = (len + c + P - 1) / P - have; }
            }
        }
        part[e] = v;
        mine = mine + v;
    }
    if (err) atomicOr(&s_err, err);
    Sums inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const Sums o{__shfl_up(inc.tok, d), __shfl_up(inc.take, d), __shfl_up(inc.give, d)};
        if (lane >= d) inc = inc + o;
    }
    if (lane == 63) wsum[wv] = inc;
    __syncthreads();
    Sums before{0, 0, 0}, all{0, 0, 0};
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w == wv) before = all;
        all = all + wsum[w];
    }
    err = s_err;
    if (all.tok > a.capacity || all.take > nfree) err |= kStNoPages;
    if (nfree - all.take + all.give > N) err |= kStPage;
    if (!err) {
        Sums run{before.tok + inc.tok - mine.tok, before.take + inc.take - mine.take, before.give + inc.give - mine.give};
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = tid * per + e;
            if (e < per && i < B) {
                s_tok[i] = (int)run.tok;
                s_take[i] = (int)run.take;
                s_give[i] = (int)run.give;
                run = run + part[e];
            }
        }
        if (tid == 0) {
            s_tok[B] = (int)all.tok;
            s_take[B] = (int)all.take;
            s_give[B] = (int)all.give;
        }
    }
    __syncthreads();

    const long long step = (long long)gridDim.x * kThreads, first = (long long)blockIdx.x * kThreads + tid;
    auto at_ring = [&](long long i) { return i >= N ? i - N : i; };
    if (err) {   // the whole step is refused
        for (long long t = first; t < a.capacity; t += step) a.slots[t] = a.positions[t] = a.rows[t] = -1;
        for (long long i = first; i <= B; i += step) a.starts[i] = 0;
        if (first == 0) atomicOr(a.status, err);
    } else {
        uint32_t bad = 0;
        for (long long t = first; t < a.capacity; t += step) {
            int slot = -1, pos = -1, row = -1;
            if (t < all.tok) {
                row = owner_of(s_tok, B, (int)t);
                const int len = a.lens[row];
                pos = len + (int)t - s_tok[row];
                const int have = (len + P - 1) / P, col = pos / P;
                const int page = col < have ? a.block_table[row * a.table_stride + col]
                                            : a.ring[at_ring(head + s_take[row] + col - have)];
                if (page >= 0 && page < N) slot = page * P + pos % P;
                else bad = kStPage;
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
            a.rows[t] = row;
        }
        for (long long i = first; i <= B; i += step) a.starts[i] = s_tok[i];
        for (long long p = first; p < all.take; p += step) {
            const int i = owner_of(s_take, B, (int)p);
            const int have = (a.lens[i] + P - 1) / P;
            a.block_table[i * a.table_stride + have + (int)p - s_take[i]] = a.ring[at_ring(head + p)];
        }
        for (long long p = first; p < all.give; p += step) {
            const int i = owner_of(s_give, B, (int)p);
            const int page = a.block_table[i * a.table_stride + (int)p - s_give[i]];
            if (page < 0 || page >= N) bad = kStPage;
            a.ring[at_ring(at_ring(head + nfree) + p)] = page;
        }
        if (bad) atomicOr(a.status, bad);
    }

    // The last block to come here writes what the others have read.
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(reinterpret_cast<unsigned *>(a.state + 2), 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int i = tid; i < B; i += kThreads) {
        const int len = a.lens[i], c = a.counts[i];
        a.lens_out[i] = err ? len : c < 0 ? 0 : len + c;
    }
    if (tid == 0) {
        a.state[2] = 0;
        a.state_out[0] = (int)(err ? head : at_ring(head + all.take));
        a.state_out[1] = (int)(err ? nfree : nfree - all.take + all.give);
        if (a.state_out != a.state) a.state_out[2] = a.state_out[3] = 0;
    }
}

}  // namespace

hipError_t launch_kv_tables(const ikbo_kv_tables_args &a, hipStream_t s) {
    // A block's own sums cost as much as several rows for each of its threads; few blocks do.
    const long long items = (long long)a.capacity + a.B_u;
    const int blocks = (int)std::min<long long>(256, std::max<long long>(1, (items + 2 * kThreads - 1) / (2 * kThreads)));
    const size_t lds = 3 * (size_t)(a.B_u + 1) * sizeof(int);   // at most 48 KB
    hipLaunchKernelGGL(kv_tables_kernel, dim3(blocks), dim3(kThreads), lds, s, a);
    return hipGetLastError();
}

}  // namespace ikbo
