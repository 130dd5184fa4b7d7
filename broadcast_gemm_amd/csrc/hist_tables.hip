// hist_tables.hip -- page tables, slots, positions and rows of one step (ikbo_kv_tables).
//
// With the exclusive prefix sums over the requests of new tokens (starts), pages taken and pages
// returned, every output has a closed form: token row t belongs to the request i with
// starts[i] <= t < starts[i+1]; page p of the taken ones is ring[head + p] and opens with the token at
// its first place, which also enters it in the table; page p of the returned ones belongs to the request
// whose range of the third sum holds p.  So no block needs another's result: each block forms the
// three sums itself (at most 4096 requests, 4 per thread, one block-wide scan) and then takes its share
// of the rows and pages, found by binary search in LDS.  One launch, no waiting between blocks; what it
// costs is the chain of a few dependent reads (3.9 us for a step of 59 requests, 10.4 us for 4096 requests with 65000
// tokens, of which the scan of the counts and the searches are most).
//
// In-place lengths and ring state may only change once every block has read them: a block counts
// itself in state[2] when it is done, and the last one writes lens_out and state_out and sets the
// count back to 0 (out of place the first block writes them at once).  The ring's popped and pushed
// places are disjoint (a step whose returned pages and free ones are more than the ring is refused), and so are the table entries read (the page a
// request's next token falls into) and written (the ones behind it): those are updated where they are.
//
// The sums saturate at 2^32 - 1: that is more than any capacity or ring, so a step that reaches it is
// refused whatever the true sum is.
#include "hist_internal.h"

#include <algorithm>

namespace ikbo {
namespace {

constexpr int kMost = 1024;                          // threads of a block, at most
constexpr int kPer = IKBO_KV_MAX_USERS / kMost;      // requests per thread

struct Sums {
    uint32_t tok, take, give;
};

__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }
__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) { return {add(a.tok, b.tok), add(a.take, b.take), add(a.give, b.give)}; }

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

__global__ void __launch_bounds__(kMost) kv_tables_kernel(ikbo_kv_tables_args a) {
    extern __shared__ int sh[];
    const int B = a.B_u, P = a.page_size, N = a.num_pages, nt = (int)blockDim.x;
    int *s_tok = sh, *s_take = sh + B + 1, *s_give = sh + 2 * (B + 1), *s_len = sh + 3 * (B + 1);
    __shared__ Sums wsum[kMost / 64];
    __shared__ uint32_t werr[kMost / 64];
    __shared__ int s_last;
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;

    // Each thread sums its consecutive requests, then a scan over the threads.
    const int per = (B + nt - 1) / nt;
    int len[kPer], cnt[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = tid * per + e;
        const bool mine = e < per && i < B;
        len[e] = mine ? a.lens[i] : 0;
        cnt[e] = mine ? a.counts[i] : 0;
    }
    const int head = a.state[0], nfree = a.state[1];
    const long long most = (long long)a.max_pages * P;
    Sums mine{0, 0, 0}, part[kPer];
    uint32_t err = head < 0 || head >= N || nfree < 0 || nfree > N ? kStPage : 0u;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        Sums v{0, 0, 0};
        if (len[e] < 0 || len[e] > most || cnt[e] < -1) err |= kStPage;
        else if (len[e] + (long long)cnt[e] > most) err |= kStNoPages;
        else {
            const uint32_t have = ((uint32_t)len[e] + P - 1) / P;
            if (cnt[e] < 0) v.give = have;
            else { v.tok = cnt[e]; v.take = ((uint32_t)len[e] + cnt[e] + P - 1) / P - have; }
        }
        part[e] = v;
        mine = mine + v;
    }
    Sums inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const Sums o{__shfl_up(inc.tok, d), __shfl_up(inc.take, d), __shfl_up(inc.give, d)};
        if (lane >= d) inc = inc + o;
    }
    if (lane == 63) wsum[wv] = inc;
    const uint32_t any = (__ballot(err & kStPage) ? kStPage : 0u) | (__ballot(err & kStNoPages) ? kStNoPages : 0u);
    if (lane == 0) werr[wv] = any;
    __syncthreads();
    Sums before{0, 0, 0}, all{0, 0, 0};
    err = 0;
    for (int w = 0; w < nt / 64; ++w) {
        if (w == wv) before = all;
        all = all + wsum[w];
        err |= werr[w];
    }
    if (all.tok > (uint32_t)a.capacity || all.take > (uint32_t)nfree) err |= kStNoPages;
    // Free pages and those that lengths hold are N at most.  With more (a page returned twice, a length overstated) the
    // pushed places would reach round the ring into the popped ones.
    if ((long long)nfree + all.give > N) err |= kStPage;
    if (!err) {   // then no sum has saturated
        Sums run{before.tok + inc.tok - mine.tok, before.take + inc.take - mine.take, before.give + inc.give - mine.give};
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = tid * per + e;
            if (e < per && i < B) {
                s_tok[i] = (int)run.tok;
                s_take[i] = (int)run.take;
                s_give[i] = (int)run.give;
                s_len[i] = len[e];
                run = run + part[e];
            }
        }
        if (tid == 0) s_tok[B] = (int)all.tok;
    }
    __syncthreads();

    auto commit = [&] {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = tid * per + e;
            if (e < per && i < B) a.lens_out[i] = err ? len[e] : cnt[e] < 0 ? 0 : len[e] + cnt[e];
        }
        if (tid == 0) {
            const long long h = (long long)head + all.take;
            a.state[2] = 0;
            a.state_out[0] = err ? head : (int)(h >= N ? h - N : h);
            a.state_out[1] = (int)(err ? nfree : nfree - all.take + all.give);
            if (a.state_out != a.state) a.state_out[2] = a.state_out[3] = 0;
        }
    };
    const bool in_place = a.lens_out == a.lens || a.lens_out == a.counts || a.state_out == a.state;
    if (!in_place && blockIdx.x == 0) commit();

    const long long step = (long long)gridDim.x * nt, first = (long long)blockIdx.x * nt + tid;
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
                const int n = s_len[row];
                pos = n + (int)t - s_tok[row];
                const int have = (int)(((uint32_t)n + P - 1) / P), col = pos / P;
                int32_t *entry = a.block_table + row * a.table_stride + col;
                const int page = col < have ? *entry : a.ring[at_ring((long long)head + s_take[row] + col - have)];
                if (pos - col * P == 0) *entry = page;   // the page's first token
                if (page >= 0 && page < N) slot = page * P + pos - col * P;
                else bad = kStPage;
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
            a.rows[t] = row;
        }
        for (long long i = first; i <= B; i += step) a.starts[i] = s_tok[i];
        for (long long p = first; p < all.give; p += step) {
            const int i = owner_of(s_give, B, (int)p);
            const int page = a.block_table[i * a.table_stride + (int)p - s_give[i]];
            if (page < 0 || page >= N) bad = kStPage;
            a.ring[at_ring(at_ring((long long)head + nfree) + p)] = page;
        }
        if (bad) atomicOr(a.status, bad);
    }

    // In place, the last block to come here writes what the others have read (their reads are complete: they
    // went into what they have stored).
    if (!in_place) return;
    __syncthreads();
    if (tid == 0)
        s_last = __hip_atomic_fetch_add(reinterpret_cast<unsigned *>(a.state + 2), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    __syncthreads();
    if (s_last) commit();
}

}  // namespace

hipError_t launch_kv_tables(const ikbo_kv_tables_args &a, hipStream_t s) {
    // Small blocks scan sooner; every block repeats the scan, which costs what a row's chain of reads does.
    const int threads = a.B_u <= 1024 ? 256 : kMost;
    const long long items = std::max<long long>(a.capacity, a.B_u + 1);
    const int blocks = (int)std::min<long long>(256, std::max<long long>(1, (items + threads - 1) / threads));
    const size_t lds = 4 * (size_t)(a.B_u + 1) * sizeof(int);   // at most 64 KB and 16 bytes
    if (lds > 60 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kv_tables_kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 66 * 1024);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kv_tables_kernel, dim3(blocks), dim3(threads), lds, s, a);
    return hipGetLastError();
}

}  // namespace ikbo
