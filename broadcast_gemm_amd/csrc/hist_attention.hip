// hist_attention.hip -- target attention over the 4-bit paged cache (ikbo_kv4_attention).
//
// For one user and one key/value head, every query row of the user's candidates (candidate, query,
// head of the group) multiplies the same cached K and V: the rows stand beside one another in the
// matrix operands, 16 to a tile, and the cache is read once for all of them, never per candidate.
//
// Per page of 64 tokens a wave forms S^T = K Q^T and O^T += V^T P^T with v_mfma_f32_16x16x32_bf16.
// The hardware's 4-bit conversion applies a block's scale as it converts, and all its results are
// exact in bf16.  With lane = 16 g + j:
//   S^T tile t (A: keys, B: queries): row j of the tile is token 16 (j / 4) + 4 t + j % 4, so lane
//   (g, j) ends up with query j against tokens 16 g + 4 t + i, i < 4: over the four tiles 16
//   consecutive tokens, 16 g .. 16 g + 15.  Those are the k slots that it must supply as B operand
//   P^T, and the tokens of its A operand V^T: 16 consecutive bytes of a row of the tile's V codes.
//   The d order of the S^T product is free as long as K and Q agree.
//   A byte of V codes holds elements 2c, 2c + 1 of one token: the low halves of the converted pairs
//   belong to the even element's row of V^T, the high halves to the odd one's.
// The running maximum is kept per query; it moves (and O^T is rescaled) only when a page's maximum
// exceeds it by more than 8 (in base 2), so weights stay below 2^8.  Weights are rounded to bf16 for
// the product, and their sums are sums of the rounded ones (an all-ones A operand): half a step of
// bf16 on a weight, as in the dense attention.
//
// The wide kernel does the same with v_mfma_f32_32x32x16_bf16 and lane = 32 g + j: row j of tile t is token 32 t +
// j with bits 2 and 3 exchanged, and the lane ends up with tokens 16 s + 8 g + i, i < 8, for its four steps s.  Half
// the matrix instructions leave more room for vector work beside them: head 128 205 -> 202 us, head 64 101 -> 94.
//
// Two kernels.  In the narrow one a block is one wave with 16 or 32 rows, which converts the codes it
// reads for itself, registers to registers: with few rows the cache's bytes are what counts, and 8 waves
// on a CU keep 5 TB/s and more of them coming (0.46 GB of histories, one token each: 78-81 us, 5.7 TB/s).
// Every wave repeats the conversion, so with many rows per user and head a block of 8 waves, 32 rows each,
// converts a page once into LDS (bf16) and each wave reads its operands there.  What bounds it is the sum of
// its parts, which two waves on a SIMD overlap only in part: of 1.83 us per page of 256 rows at head 128 (1.2
// PFLOP/s) the matrix instructions take 0.95 at full rate, the softmax's and the conversion's vector work 0.95, LDS
// 0.6; to begin and end a piece of a unit takes 5.9 us.  1024 candidates of 64 rows (123 GFLOP): 158 us, 775 TFLOP/s.
// These are of a device whose clock is up, which takes some hundred passes; where two variants are compared below and in
// hist_plan.h, both were timed over the first 20, in which this launch takes 184 us.
//
// How the work is dealt to the blocks, and what joins their partial results: hist_plan.h.
#include <algorithm>

#include "hist_plan.h"
#include "lce_device.h"
#include "lce_sync.h"

namespace ikbo {
namespace {

constexpr int kLogNarrow = 11;        // one wave each, 8 at a time on each of 256 CUs
constexpr int kLogWide = 8;           // 8 waves each, one at a time on each CU
constexpr int kBuffers = 4;           // pages in LDS (wide kernel)
constexpr float kSlack = 8.0f;

// One block.  Groups the candidates by user (perm, off: a stable counting sort, one run of
// candidates per wave) and forms the prefix sums of the plan.
__global__ void __launch_bounds__(kPrep) kv4_prep_kernel(AttnArgs a, int waves) {
    extern __shared__ int sh[];       // counts [waves][B_u], offsets [B_u + 1]
    __shared__ int64_t s_w[kPrep / 64];
    __shared__ int s_n[kPrep / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int B = a.B_u;
    int *cnt = sh, *offs = sh + waves * B;
    uint32_t err = 0;
    const int per = (B + kPrep - 1) / kPrep;   // consecutive users per thread
    int len[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) len[e] = e < per && tid * per + e < B ? a.lens[tid * per + e] : 0;

    if (a.map) {
        for (int i = tid; i < waves * B; i += kPrep) cnt[i] = 0;
        __syncthreads();
        const int seg = ((a.B_c + waves - 1) / waves + 63) / 64 * 64;
        const int lo = wv * seg, hi = min(a.B_c, lo + seg);
        // One wave's candidates, 64 at a time: each distinct user among them once.
        auto walk = [&](auto each) {
            if (wv < waves)
                for (int b0 = lo, next = lo + lane < hi ? a.map[lo + lane] : -1; b0 < hi; b0 += 64) {
                    const int b = b0 + lane, u = next;
                    next = b + 64 < hi ? a.map[b + 64] : -1;
                    const bool valid = u >= 0 && u < B;
                    if (!valid && u != -1) err = kStMap;
                    uint64_t rem = __ballot(valid);
                    while (rem) {
                        const int lu = __shfl(u, __ffsll((unsigned long long)rem) - 1);
                        const uint64_t m = __ballot(valid && u == lu);
                        each(b, lu, valid && u == lu, m);
                        rem &= ~m;
                    }
                }
        };
        walk([&](int, int u, bool, uint64_t m) {
            if (lane == 0) cnt[wv * B + u] += __popcll(m);
        });
        __syncthreads();
        int sum = 0, all;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int u = tid * per + e;
            if (e < per && u < B) {
                int run = 0;
                for (int w = 0; w < waves; ++w) {
                    const int c = cnt[w * B + u];
                    cnt[w * B + u] = run;
                    run += c;
                }
                offs[u] = run;
                sum += run;
            }
        }
        int at = wave_before(sum, &all);
        if (lane == 0) s_n[wv] = all;
        __syncthreads();
        for (int w = 0; w < wv; ++w) at += s_n[w];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int u = tid * per + e;
            if (e < per && u < B) {
                const int c = offs[u];
                offs[u] = at;
                at += c;
                if (u == B - 1) offs[B] = at;
            }
        }
        __syncthreads();
        walk([&](int b, int u, bool mine, uint64_t m) {
            int first = 0;
            if (lane == 0) {
                first = cnt[wv * B + u];
                cnt[wv * B + u] = first + __popcll(m);
            }
            first = __shfl(first, 0);
            if (mine) a.perm[offs[u] + first + __popcll(m & ((1ull << lane) - 1))] = b;
        });
    } else {
        for (int b = tid; b < a.B_c; b += kPrep) a.perm[b] = b;
        for (int u = tid; u <= B; u += kPrep) offs[u] = min(u, a.B_c);
        __syncthreads();
    }
    for (int u = tid; u <= B; u += kPrep) a.off[u] = offs[u];

    int64_t w[kPer], sum_w = 0, all_w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        const int rows = e < per && u < B ? (offs[u + 1] - offs[u]) * a.L_q * a.G : 0;
        if (len[e] < 0 || len[e] > a.max_pages * kPage) err |= kStPage;
        w[e] = (int64_t)((rows + a.R - 1) / a.R) * a.H_kv * max(1, pages_of(clamp_len(len[e], a.max_pages)));
        sum_w += w[e];
    }
    int64_t at_w = wave_before(sum_w, &all_w);
    if (lane == 0) s_w[wv] = all_w;
    __syncthreads();
    all_w = 0;
    for (int v = 0; v < kPrep / 64; ++v) {
        if (v == wv) at_w += all_w;
        all_w += s_w[v];
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        if (e < per && u < B) {
            a.work[u] = at_w;
            at_w += w[e];
        }
    }
    if (tid == 0) {
        a.work[B] = all_w;
        a.share[0] = share_of(all_w, a.log_blocks);
    }
    if (err) atomicOr(a.status, err);
}

// x against the lanes 32 away, and 16 away where a group is 16 lanes.
template <int W>
__device__ __forceinline__ float max_over_groups(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const float y = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
    if constexpr (W == 32) return y;
    const uint32_t c = __builtin_bit_cast(uint32_t, y);
    const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)q[0]), __builtin_bit_cast(float, (uint32_t)q[1]));
}

// Byte i of w as a power-of-two scale: the conversion reads the exponent field alone, so the
// neighbouring bytes may stand in the sign and mantissa.
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
    return __builtin_bit_cast(float, i == 0 ? w << 23 : i == 1 ? w << 15 : i == 2 ? w << 7 : w >> 1);
}

template <int I>
__device__ __forceinline__ uint32_t values2(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
}

// The 8 values of one dword of codes of one token.
__device__ __forceinline__ u32x4_t values8(uint32_t codes, float scale) {
    return (u32x4_t){values2<0>(codes, scale), values2<1>(codes, scale), values2<2>(codes, scale), values2<3>(codes, scale)};
}

// One element pair of 4 tokens: the even element's values, then the odd one's.
__device__ __forceinline__ void values_v(uint32_t codes, uint32_t scales, uint32_t &e0, uint32_t &e1, uint32_t &o0, uint32_t &o1) {
    const uint32_t v0 = values2<0>(codes, scale_of(scales, 0)), v1 = values2<1>(codes, scale_of(scales, 1));
    const uint32_t v2 = values2<2>(codes, scale_of(scales, 2)), v3 = values2<3>(codes, scale_of(scales, 3));
    e0 = pair16(v0, v1, false);
    e1 = pair16(v2, v3, false);
    o0 = pair16(v0, v1, true);
    o1 = pair16(v2, v3, true);
}

// V scales of 4 tokens of which the first n exist.  Bytes past the history may be anything: scale
// 2^-127 keeps their values finite, and their weights are 0.
__device__ __forceinline__ uint32_t existing(uint32_t scales, int n) {
    return n >= 4 ? scales : n <= 0 ? 0u : scales & ((1u << (8 * n)) - 1u);
}

__device__ __forceinline__ float inverse_of(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }   // a row that sees nothing is 0
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

using ikbo::mfma_bf16;
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 32x32x16 bf16 MFMA: lane (g, j) = 32 g + j supplies A[j][8 g ..] and B[8 g ..][j]; acc[i] of it is D[8 (i / 4) + 4 g + i % 4][j].
__device__ __forceinline__ f32x16_t mfma_bf16(const u32x4_t &a, const u32x4_t &b, f32x16_t acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
}

// Bytes in device memory, said to the compiler: an address put together from integers is a flat one to it otherwise,
// and the wait for an LDS read then waits for every such load in flight as well.  ONCE: not to be kept in the caches.
typedef const __attribute__((address_space(1))) char *global_bytes;
template <class T, bool ONCE = false>
__device__ __forceinline__ T load_global(global_bytes p) {
    const auto x = (const __attribute__((address_space(1))) T *)p;
    return ONCE ? __builtin_nontemporal_load(x) : *x;
}

// A wave's query rows, W n + j from `first`, and their softmax: NT tiles of W rows, on the W x W matrix instruction;
// lane = W g + j.  Of a page's scores a lane holds EACH per query, element e (S[e / ACC][n][e % ACC]) being that of
// token W/2 (e / 8) + 8 g + e % 8 with W = 32, 16 g + e with W = 16.
template <int HD, int NT, int W>
struct Queries {
    static constexpr int TK = HD * W / 512, DT = HD / W, ACC = W * W / 64, TILES = kPage / W, EACH = TILES * ACC, STEPS = EACH / 8;
    typedef float acc_t __attribute__((ext_vector_type(ACC)));
    int limit[NT];                    // tokens that the row sees
    int most, least;                  // largest and smallest limit of the wave's rows
    u32x4_t qf[TK][NT];
    acc_t o[DT][NT], lsum[NT];
    float m[NT], nm[NT];

    static __device__ __forceinline__ int token(int e, int g) { return W == 16 ? 16 * g + e : 16 * (e >> 3) + 8 * g + (e & 7); }

    const uint16_t *from[NT];         // the rows in Q
    int64_t to[NT];                   // and in O
    int pos[NT];
    bool live[NT];

    template <class P>
    __device__ __forceinline__ void find(const AttnArgs &a, const P &plan, const User &x, int h, int first, int j) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = first + W * n + j;
            live[n] = r < x.n_rows;
            int cnd, l, hq;
            plan.row(x, h, live[n] ? r : 0, cnd, l, hq);
            from[n] = a.Q + cnd * a.q_cand + hq * a.q_head + l * a.q_query;
            to[n] = cnd * a.o_cand + hq * a.o_head + l * a.o_query;
            if (a.positions) pos[n] = load_global<int32_t>((global_bytes)a.positions + 4 * ((int64_t)cnd * a.L_q + l));
        }
    }
    // Step s of a row's elements: lane group g holds the 8 from `base` + s * `step`.
    __device__ __forceinline__ void load(const AttnArgs &a, const User &x, int base, int step) {
        most = least = x.len;
        if (a.positions) most = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int s = 0; s < TK; ++s)
                qf[s][n] = live[n] ? *reinterpret_cast<const u32x4_t *>(from[n] + base + s * step) : (u32x4_t){0, 0, 0, 0};
            limit[n] = live[n] ? x.len : 0;
            if (live[n] && a.positions) limit[n] = pos[n] < 0 ? 0 : pos[n] < x.len ? pos[n] + 1 : x.len;
        }
        if (a.positions) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                most = max(most, limit[n]);
                if (live[n]) least = min(least, limit[n]);
            }
#pragma unroll
            for (int d = 1; d < W; d <<= 1) {
                most = max(most, __shfl_xor(most, d));
                least = min(least, __shfl_xor(least, d));
            }
            most = __builtin_amdgcn_readfirstlane(most);
            least = __builtin_amdgcn_readfirstlane(least);
        }
    }

    __device__ __forceinline__ void start() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -__builtin_inff();
            nm[n] = 0.f;
            lsum[n] = (acc_t)(0.f);
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d][n] = (acc_t)(0.f);
        }
    }

    // Scores of page p: what a row does not see becomes -inf, and the running maximum moves if it must.
    __device__ __forceinline__ void raise(acc_t (&S)[TILES][NT], int p, int g, float scale_log2) {
        // The empty asm keeps these two branches branches: their bodies cost more than a turn's own
        // vector work, and as selects they would be paid on every page.
        if (p * kPage + kPage > least) {
            asm volatile("");
            const int key0 = p * kPage + token(0, g);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < EACH; ++e)
                    if (key0 + token(e, 0) >= limit[n]) S[e / ACC][n][e % ACC] = -__builtin_inff();
        }
        bool grow = false;
        float mb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x = -__builtin_inff();
#pragma unroll
            for (int e = 0; e < EACH; ++e) x = fmaxf(x, S[e / ACC][n][e % ACC]);
            mb[n] = max_over_groups<W>(x) * scale_log2;
            grow = grow || mb[n] > m[n] + kSlack;
        }
        if (__ballot(grow)) {
            asm volatile("");
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float mn = fmaxf(m[n], mb[n]);
                const float alpha = mn == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                m[n] = mn;
                nm[n] = mn == -__builtin_inff() ? 0.f : -mn;
                lsum[n] *= alpha;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d][n] *= alpha;
            }
        }
    }

    // Scores into the weights pf (B operand of the steps of 512 / W tokens) and their sums, steps [s0, s1).
    __device__ __forceinline__ void weigh(const acc_t (&S)[TILES][NT], float scale_log2, u32x4_t (&pf)[STEPS][NT], int s0 = 0, int s1 = STEPS) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 8 * s0; e < 8 * s1; e += 4) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[e / ACC][n][e % ACC + i], scale_log2, nm[n]));
                pf[e >> 3][n][(e & 7) >> 1] = pack_bf16x2(w[0], w[1]);
                pf[e >> 3][n][((e & 7) >> 1) + 1] = pack_bf16x2(w[2], w[3]);
            }
        const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
        for (int s = s0; s < s1; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) lsum[n] = mfma_bf16(ones, pf[s][n], lsum[n]);
    }
};

// A run of the line of pages: the pieces of units that block `blk` takes, one after the other.
struct Piece {
    User x;
    int h, tile, p0, p1;
    bool whole;
    int64_t slot;                     // of the partial result, unless whole
    int n;                            // pieces of the unit, if it begins here and is cut
};
// Where the run of block `blk` begins (that of block `blk` - 1 ends).
template <class P>
__device__ __forceinline__ int64_t edge_of(const AttnArgs &a, const P &plan, int64_t blk) {
    const int64_t all = plan.work[a.B_u], x = blk * plan.share, near = near_of(plan.share);
    if (x <= 0) return 0;
    if (x >= all) return all;
    const int u = owner_of(plan.work, a.B_u, x);
    const int64_t pages = plan.pages_of_user(u), in_u = x - plan.work[u], in = in_u - over(in_u, pages) * pages;
    if (in <= near && in <= pages - in) return x - in;
    return pages - in <= near ? x + pages - in : x;
}
template <class P>
__device__ __forceinline__ Piece piece_at(const AttnArgs &a, P &plan, User &x, int64_t at, int64_t end, int64_t blk) {
    Piece c;
    if (at >= x.to) x = plan.enter(owner_of(plan.work, a.B_u, at));   // most runs stay with one user
    c.x = x;
    // Within a user units and pages are counted in 64 bits; a unit's number fits 32.
    const int64_t local = at - c.x.from;
    const int64_t unit = over(local, c.x.pages);
    c.p0 = (int)(local - unit * c.x.pages);
    c.p1 = (int)min((int64_t)c.x.pages, c.p0 + (end - at));
    c.h = (int)((uint32_t)unit / (uint32_t)c.x.tiles);
    c.tile = (int)unit - c.h * c.x.tiles;
    c.whole = c.p0 == 0 && c.p1 == c.x.pages;
    c.slot = 2 * blk + (c.p0 == 0);
    // The pieces end at the runs' ends that lie further than `near` from both edges of the unit.
    const int64_t near = near_of(plan.share);
    c.n = c.p0 == 0 && !c.whole ? (int)(over(at + c.x.pages - near - 1, plan.share) - over(at + near, plan.share)) + 1 : 0;
    return c;
}

// Blocks are dealt to the 8 dies in turn: give each die neighbouring runs, whose units share K and V.
__device__ __forceinline__ int64_t run_of_block(int blocks) {
    return (blocks & 7) ? blockIdx.x : (int64_t)(blockIdx.x & 7) * (blocks >> 3) + (blockIdx.x >> 3);
}

// The tiles of a run of pages: lane i keeps the page number of page base + i, so that a tile's address
// needs no load of its own (64 pages at a time; a wait on the table in every turn cost the wide kernel
// a third of its time).
struct Pages {
    global_bytes row;
    const char *tiles;                // head h of page 0
    int64_t stride;                   // bytes from page to page
    int user = -1, base, end, last, num_pages, ids;
    bool bad;
    __device__ __forceinline__ void open(const AttnArgs &a, const Piece &c, int tile_bytes) {
        tiles = a.tiles + (int64_t)c.h * tile_bytes;
        stride = (int64_t)a.H_kv * tile_bytes;
        num_pages = a.num_pages;
        // Entries behind the history may hold anything; an empty one has none.
        end = pages_of(c.x.len) - 1;
        last = min(c.p1 - 1, end);
        bad = false;
        if (c.x.u == user && c.p0 >= base && c.p0 - base < 64) return;   // a unit of the same user: the numbers are here
        user = c.x.u;
        row = (global_bytes)(a.table + (int64_t)user * a.table_stride);
        base = 0;
        ids = 0;
        if (c.p0 <= last) read(c.p0);
    }
    __device__ __forceinline__ void read(int p) {
        base = p;
        ids = load_global<int32_t>(row + 4 * (int64_t)min(p + ((int)threadIdx.x & 63), end));
    }
    // The tile of page p (of the last page if p is behind it); p never decreases by more than the caller's look-ahead.
    __device__ __forceinline__ global_bytes at(int p) {
        p = min(p, last);
        if (p - base >= 64) read(p);
        int page = __builtin_amdgcn_readlane(ids, p - base);
        if (page < 0 || page >= num_pages) { bad = true; page = 0; }
        // In scalar registers: loads then take it as their base.
        const uint64_t at = reinterpret_cast<uint64_t>(tiles) + (uint64_t)page * stride;
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
        return (global_bytes)(((uint64_t)hi << 32) | lo);
    }
};

// What a lane reads of a page.
template <int HD>
struct PageRegs {
    static constexpr int KW = HD / 32;     // dwords of a K row per lane
    static constexpr int VJ = HD / 32;     // 16-pair groups of V rows
    uint32_t k[4][KW];
    uint32_t ks;
    u32x4_t v[VJ], vs[VJ];
    template <bool ONCE>
    __device__ __forceinline__ void load_k(global_bytes tile, int g, int j) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const global_bytes p = tile + (16 * (j >> 2) + 4 * t + (j & 3)) * (HD / 2) + g * (HD / 8);
            if constexpr (HD == 128) {
                const u32x4_t w = load_global<u32x4_t, ONCE>(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) k[t][i] = w[i];
            } else {
                const u32x2_t w = load_global<u32x2_t, ONCE>(p);
                k[t][0] = w[0];
                k[t][1] = w[1];
            }
        }
        ks = load_global<uint32_t, ONCE>(tile + 64 * HD + (HD == 128 ? g : g >> 1) * 64 + 4 * j);
    }
    template <bool ONCE>
    __device__ __forceinline__ void load_v(global_bytes tile, int g, int j) {
#pragma unroll
        for (int jj = 0; jj < VJ; ++jj) {
            v[jj] = load_global<u32x4_t, ONCE>(tile + 32 * HD + (16 * jj + j) * 64 + 16 * g);
            vs[jj] = load_global<u32x4_t, ONCE>(tile + 66 * HD + jj * 64 + 16 * g);
        }
    }
};

template <int HD, int NT, bool SMALL, bool ONCE>
__global__ void __launch_bounds__(64, 2) kv4_attn_kernel(AttnArgs a) {
    constexpr int VJ = HD / 32, TILE = 68 * HD;
    __shared__ PlanLds<SMALL> small;
    const int lane = (int)threadIdx.x, g = lane >> 4, j = lane & 15;
    Plan<SMALL, 64> plan(a, small);
    const int64_t blk = run_of_block((int)gridDim.x), end = edge_of(a, plan, blk + 1);
    int2 note = make_int2(0, 0);
    User user;
    user.to = -1;
    Pages pages;
    for (int64_t at = edge_of(a, plan, blk); at < end;) {
        const Piece c = piece_at(a, plan, user, at, end, blk);
        if (c.n) note = make_int2(c.n, min(a.R, c.x.n_rows - c.tile * a.R));
        at += c.p1 - c.p0;
        pages.open(a, c, TILE);   // the table's entries are on their way while the queries are found
        Queries<HD, NT, 16> q;
        // The d order of K and Q: lane group g takes the g-th quarter of a head, one piece of a K row.
        q.find(a, plan, c.x, c.h, c.tile * 16 * NT, j);
        q.load(a, c.x, g * (HD / 4), 8);
        q.start();
        const int p1 = min(c.p1, (q.most + kPage - 1) / kPage);   // no row sees further pages
        PageRegs<HD> pg;
        for (int p = c.p0; p < p1; ++p) {
            const global_bytes tile = pages.at(p);
            pg.template load_k<ONCE>(tile, g, j);
            pg.template load_v<ONCE>(tile, g, j);
            f32x4_t S[4][NT];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float ks = scale_of(pg.ks, t);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[t][n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < HD / 32; ++s) {
                    const u32x4_t kf = values8(pg.k[t][s], ks);
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[t][n] = mfma_bf16(kf, q.qf[s][n], S[t][n]);
                }
            }
            if (p * kPage + kPage > c.x.len) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int jj = 0; jj < VJ; ++jj) pg.vs[jj][t] = existing(pg.vs[jj][t], c.x.len - (p * kPage + 16 * g + 4 * t));
            }
            u32x4_t pf[2][NT];
            q.raise(S, p, g, a.scale_log2);
            q.weigh(S, a.scale_log2, pf);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    u32x4_t even, odd;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t e0, e1, o0, o1;
                        values_v(pg.v[jj][2 * kk + y], pg.vs[jj][2 * kk + y], e0, e1, o0, o1);
                        even[2 * y] = e0;
                        even[2 * y + 1] = e1;
                        odd[2 * y] = o0;
                        odd[2 * y + 1] = o1;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        q.o[2 * jj][n] = mfma_bf16(even, pf[kk][n], q.o[2 * jj][n]);
                        q.o[2 * jj + 1][n] = mfma_bf16(odd, pf[kk][n], q.o[2 * jj + 1][n]);
                    }
                }
        }
        if (pages.bad && lane == 0) atomicOr(a.status, kStPage);

        // Lane (g, j) holds of query j the elements 32 jj + 8 g + 2 i (even tile) and + 1 (odd tile).
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int in_unit = 16 * n + j, r = c.tile * 16 * NT + in_unit;
            if (r >= c.x.n_rows) continue;
            const float l = q.lsum[n][0];
            const int64_t o_at = q.to[n];
            if (c.n && g == 0) a.note_o[blk * a.R + in_unit] = o_at;
            if (c.whole) {
                const float inv = inverse_of(l);
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    u32x4_t w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(q.o[2 * jj][n][i] * inv, q.o[2 * jj + 1][n][i] * inv);
                    *reinterpret_cast<u32x4_t *>(a.O + o_at + 32 * jj + 8 * g) = w;
                }
            } else {
                const int64_t to = c.slot * (16 * NT) + in_unit;
                if (g == 0) a.ml[to] = make_float2(q.m[n], l);
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    f32x4_t w0, w1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        w0[2 * i] = q.o[2 * jj][n][i];
                        w0[2 * i + 1] = q.o[2 * jj + 1][n][i];
                        w1[2 * i] = q.o[2 * jj][n][2 + i];
                        w1[2 * i + 1] = q.o[2 * jj + 1][n][2 + i];
                    }
                    *reinterpret_cast<f32x4_t *>(a.part + to * HD + 32 * jj + 8 * g) = w0;
                    *reinterpret_cast<f32x4_t *>(a.part + to * HD + 32 * jj + 8 * g + 4) = w1;
                }
            }
        }
    }
    if (lane == 0) a.note[blk] = note;
}

// ---- the wide kernel -----------------------------------------------------------------------

// Four page buffers in LDS: K rows [64 tokens][HD] and V^T rows [HD][64 tokens], bf16.  The 16-byte chunks of a row
// stand permuted by an XOR with a number of the row.  A 16-byte access of a wave is served 16 lanes at a time, and not
// in their order: lanes 0-3, 12-15, 20-23 and 24-27, then 4-11, 16-19 and 28-31, and so on (measured with pairs of
// patterns).  Those of the first set and those of the second hold each value of j % 16 once among j = lane % 32, and
// their g is the same: the 16 rows' chunks fall on 16 places of 256 bytes if the numbers are j % 16 for rows of 256
// bytes, (j / 2) % 8 for rows of 128, where neighbouring rows are the two halves.  Without conflicts a wave's read
// takes 4 cycles instead of 8 and more.
template <int HD>
struct WideLds {
    static constexpr int KBYTES = kPage * HD * 2, PAGE = 2 * KBYTES;
    // Chunk c of token `key`.
    static __device__ __forceinline__ int k_at(int key, int c) {
        const int j = (key & 19) | (key & 4) << 1 | (key & 8) >> 1;   // the token's place in the operand
        return key * HD * 2 + ((c ^ (HD == 128 ? j & 15 : (j >> 1) & 7)) << 4);
    }
    // Chunk c of element d; the rows of a pair change places with every pair, for the writes.
    static __device__ __forceinline__ int v_at(int d, int c) {
        return KBYTES + (d ^ ((d >> 1) & 1)) * kPage * 2 + ((c ^ ((d >> 1) & 7)) << 4);
    }
};

// A barrier that waits for this wave's LDS accesses only: codes in flight stay so.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
    wg_barrier();
}

template <int HD>
__global__ void __launch_bounds__(512, 1) kv4_wide_kernel(AttnArgs a) {
    typedef WideLds<HD> L;
    constexpr int WAVES = 8, ROWS = 32 * WAVES, THREADS = 64 * WAVES, TK = HD / 16, DT = HD / 32, TILE = 68 * HD;
    // 8-byte pieces of a page's K codes (and of its V codes) and how many of them a thread takes; with more
    // threads than pieces the first half of the threads takes K and the second V.
    constexpr int PIECES = kPage * HD / 16, JOBS = PIECES >= THREADS ? PIECES / THREADS : 1;
    constexpr bool BOTH = PIECES >= THREADS;
    static_assert(BOTH || 2 * PIECES == THREADS, "every thread takes K, V or both");
    extern __shared__ __align__(16) char lds[];
    __shared__ PlanLds<false> in_workspace;
    __shared__ int s_most[2][WAVES];
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6, g = lane >> 5, j = lane & 31;
    Plan<false, THREADS> plan(a, in_workspace);
    int odd_piece = 0;
    const int64_t blk = run_of_block((int)gridDim.x), end = edge_of(a, plan, blk + 1);
    int2 note = make_int2(0, 0);
    // This thread's operand reads (K tile t: + 4 t rows; V tile x: + 16 x rows), and where its pieces come from and
    // go to: K piece i is 16 elements of token i / (HD/16), V piece i 8 tokens of element pair i / 8.
    int k_off[TK], v_off[4], k_to[JOBS][2], v_to[JOBS][2], code_at[JOBS], ks_at[JOBS], vs_at[JOBS];
#pragma unroll
    for (int s = 0; s < TK; ++s) k_off[s] = L::k_at((j & 19) | (j & 4) << 1 | (j & 8) >> 1, 2 * s + g);
#pragma unroll
    for (int s = 0; s < 4; ++s) v_off[s] = L::v_at(j, 2 * s + g);
    const bool has_k = BOTH || tid < PIECES, has_v = BOTH || tid >= PIECES;
#pragma unroll
    for (int y = 0; y < JOBS; ++y) {
        const int i = (tid & (PIECES - 1)) + y * THREADS, key = i / (HD / 16), part = i % (HD / 16), pair = i >> 3;
        code_at[y] = 8 * i;
        ks_at[y] = 64 * HD + (part >> 1) * 64 + (key & 48) + 4 * (key & 3) + ((key >> 2) & 3);
        vs_at[y] = 66 * HD + (i >> 7) * 64 + 8 * (i & 7);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            k_to[y][x] = L::k_at(key, 2 * part + x);
            v_to[y][x] = L::v_at(2 * pair + x, i & 7);
        }
    }
    User user;
    user.to = -1;
    Pages pages;
    for (int64_t at = edge_of(a, plan, blk); at < end;) {
        const Piece c = piece_at(a, plan, user, at, end, blk);
        if (c.n) note = make_int2(c.n, min(a.R, c.x.n_rows - c.tile * a.R));
        at += c.p1 - c.p0;
        pages.open(a, c, TILE);
        Queries<HD, 1, 32> q;
        q.find(a, plan, c.x, c.h, c.tile * ROWS + wv * 32, j);
        const int p0 = c.p0;
        u32x2_t kc[2][JOBS], vc[2][JOBS], vs[2][JOBS];
        uint32_t ks[2][JOBS];
        auto fetch = [&](int p, int w) {
            const global_bytes tile = pages.at(p);
#pragma unroll
            for (int y = 0; y < JOBS; ++y) {
                if (has_k) {
                    kc[w][y] = load_global<u32x2_t>(tile + code_at[y]);
                    ks[w][y] = load_global<uint8_t>(tile + ks_at[y]);
                }
                if (has_v) {
                    vc[w][y] = load_global<u32x2_t>(tile + code_at[y] + 32 * HD);
                    vs[w][y] = load_global<u32x2_t>(tile + vs_at[y]);
                }
            }
        };
        auto tail = [&](int p, int w) {
            const int left = c.x.len - min(p, pages.last) * kPage;   // tokens of the page that exist
            if (left < kPage) {
                asm volatile("");
#pragma unroll
                for (int y = 0; y < JOBS; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) vs[w][y][x] = existing(vs[w][y][x], left - (8 * (tid & 7) + 4 * x));
            }
        };
        auto convert = [&](int p, int w) {
            char *to = lds + (p & (kBuffers - 1)) * L::PAGE;
#pragma unroll
            for (int y = 0; y < JOBS; ++y) {
                if (has_k) {
                    const float s = scale_of(ks[w][y], 0);
#pragma unroll
                    for (int x = 0; x < 2; ++x) *reinterpret_cast<u32x4_t *>(to + k_to[y][x]) = values8(kc[w][y][x], s);
                }
                if (has_v) {
                    u32x4_t even, odd;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t e0, e1, o0, o1;
                        values_v(vc[w][y][x], vs[w][y][x], e0, e1, o0, o1);
                        even[2 * x] = e0;
                        even[2 * x + 1] = e1;
                        odd[2 * x] = o0;
                        odd[2 * x + 1] = o1;
                    }
                    *reinterpret_cast<u32x4_t *>(to + v_to[y][0]) = even;
                    *reinterpret_cast<u32x4_t *>(to + v_to[y][1]) = odd;
                }
            }
        };
        // The first pages' codes are on their way before the queries' are waited for, and converted before the barrier
        // below (the previous piece's last reads were before its last).
        const bool any = p0 <= pages.last;
        if (any) {
            fetch(p0, 0);
            fetch(p0 + 1, 1);
        }
        q.load(a, c.x, 8 * g, 16);
        q.start();
        int *ends = s_most[odd_piece];   // two, for a wave may be a barrier ahead of one that still reads
        odd_piece ^= 1;
        if (lane == 0) ends[wv] = q.most;
        if (any) {
            tail(p0, 0);
            convert(p0, 0);
            fetch(p0 + 2, 0);
            tail(p0 + 1, 1);
            convert(p0 + 1, 1);
            fetch(p0 + 3, 1);
        }
        lds_barrier();
        int most = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) most = max(most, ends[w]);
        const int p1 = min(c.p1, (most + kPage - 1) / kPage);   // no row sees further pages
        if (p0 < p1) {
            auto scores = [&](int p, f32x16_t (&S)[2][1]) {
                const char *from = lds + (p & (kBuffers - 1)) * L::PAGE;
                S[0][0] = S[1][0] = (f32x16_t)(0.f);
#pragma unroll
                for (int s = 0; s < TK; ++s)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const u32x4_t kf = *reinterpret_cast<const u32x4_t *>(from + k_off[s] + t * 32 * HD * 2);
                        S[t][0] = mfma_bf16(kf, q.qf[s][0], S[t][0]);
                    }
            };
            auto product = [&](int p, int s, const u32x4_t (&pf)[4][1]) {
                const char *from = lds + (p & (kBuffers - 1)) * L::PAGE;
#pragma unroll
                for (int x = 0; x < DT; ++x) {
                    const u32x4_t vf = *reinterpret_cast<const u32x4_t *>(from + v_off[s] + x * 32 * kPage * 2);
                    q.o[x][0] = mfma_bf16(vf, pf[s][0], q.o[x][0]);
                }
            };
            auto accumulate = [&](int p, const f32x16_t (&S)[2][1]) {
                u32x4_t pf[4][1];
                q.weigh(S, a.scale_log2, pf, 0, 2);   // by halves: the second's weights overlap the first's products
                product(p, 0, pf);
                product(p, 1, pf);
                q.weigh(S, a.scale_log2, pf, 2, 4);
                product(p, 2, pf);
                product(p, 3, pf);
            };
            f32x16_t S[2][1];
            // Two pages a barrier: a page's buffer takes the one four pages on, two turns after the barrier behind
            // its last reads.  Pages behind the last are taken again from the last one (into buffers that nothing
            // reads), which keeps the turns free of branches.  The conversion stands behind the scores' matrix
            // instructions, which it can overlap (in front of them: 6% slower).  Waves without a row that sees
            // the page do the same work on masked scores: a branch around it cost the others a tenth.
            auto turn = [&](int p, int w) {
                tail(p + 2, w);
                scores(p, S);
                convert(p + 2, w);
                fetch(p + 4, w);
                q.raise(S, p, g, a.scale_log2);
                accumulate(p, S);
            };
            for (int p = p0; p < p1; p += 2) {
                turn(p, 0);
                if (p + 1 < p1) turn(p + 1, 1);
                lds_barrier();
            }
            if (pages.bad && tid == 0) atomicOr(a.status, kStPage);
        }

        // Lane (g, j) holds of query j the elements 32 x + 8 y + 4 g + i.  Both lanes of a query are live, or neither is.
        const int in_unit = wv * 32 + j;
        if (q.live[0]) {
            const float l = q.lsum[0][0];
            const int64_t o_at = q.to[0];
            if (c.n && g == 0) a.note_o[blk * a.R + in_unit] = o_at;
            if (c.whole) {
                const float inv = inverse_of(l);
#pragma unroll
                for (int x = 0; x < DT; ++x)
#pragma unroll
                    for (int y = 0; y < 4; y += 2) {
                        // The lanes 32 away have each other's neighbours: g = 0 takes the 8 elements of y, g = 1 those of y + 1.
                        const f32x16_t &o = q.o[x][0];
                        u32x4_t w;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const auto p = __builtin_amdgcn_permlane32_swap(pack_bf16x2(o[4 * y + 2 * i] * inv, o[4 * y + 2 * i + 1] * inv),
                                                                            pack_bf16x2(o[4 * y + 4 + 2 * i] * inv, o[4 * y + 5 + 2 * i] * inv), false, false);
                            w[i] = p[0];
                            w[2 + i] = p[1];
                        }
                        *reinterpret_cast<u32x4_t *>(a.O + o_at + 32 * x + 8 * (y + g)) = w;
                    }
            } else {
                const int64_t to = c.slot * ROWS + in_unit;
                if (g == 0) a.ml[to] = make_float2(q.m[0], l);
#pragma unroll
                for (int x = 0; x < DT; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const f32x16_t &o = q.o[x][0];
                        *reinterpret_cast<f32x4_t *>(a.part + to * HD + 32 * x + 8 * y + 4 * g) =
                            (f32x4_t){o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]};
                    }
            }
        }
    }
    if (tid == 0) a.note[blk] = note;
}

// ---- joining partial results ---------------------------------------------------------------

// O = sum_s w_s O_s / sum_s w_s l_s with w_s = 2^(m_s - max m) over the n pieces of a unit (slots: hist_plan.h).
// A block takes 16 Y rows of the unit that its note names, Y for each of its 16 half waves (a lane holds HD/32
// neighbouring elements); where there are fewer than 16, several half waves share a row's pieces.  The chain of reads
// (note, maxima, rows) is what it costs: what does not depend on the one before is asked for early, and with
// units of 256 rows a half wave takes two of them at once (140 cut units of head 128: 11.6 us, one at a time 12.4,
// four 15.3; before the early reads 14.4).
template <int HD, int Y>
__global__ void __launch_bounds__(512) kv4_join_kernel(AttnArgs a) {
    constexpr int E = HD / 32;
    typedef float vec_t __attribute__((ext_vector_type(E)));
    __shared__ vec_t s_acc[16][32];
    const int lane = (int)threadIdx.x & 63, i = lane & 31, half = (int)threadIdx.x >> 5, r_first = 16 * Y * (int)blockIdx.y;
    const int64_t b = blockIdx.x;
    const int2 note = a.note[b];
    const int n = note.x, rows = min(16 * Y, note.y - r_first);
    if (n == 0 || rows <= 0) return;
    int abreast = 1;
    while (abreast < rows && abreast < 16) abreast <<= 1;
    const int share = 16 / abreast, k0 = half / share, part = half - k0 * share;   // half waves per row
    bool live[Y];
    int64_t o_at[Y], at0[Y];
    float top[Y], l[Y];
    vec_t acc[Y];
#pragma unroll
    for (int y = 0; y < Y; ++y) {
        const int k = k0 + 16 * y;
        live[y] = k < rows;
        at0[y] = 2 * b * a.R + r_first + (live[y] ? k : 0);
        o_at[y] = live[y] ? a.note_o[b * a.R + r_first + k] : 0;
        top[y] = -__builtin_inff();
        l[y] = 0.f;
        acc[y] = (vec_t)(0.f);
    }
    auto at = [&](int y, int s) { return at0[y] + (2 * (int64_t)s + (s == 0)) * a.R; };
    // The first pieces' numbers are read once, and those of their rows are on their way meanwhile.
    float2 ml0[Y];
    vec_t part0[Y];
#pragma unroll
    for (int y = 0; y < Y; ++y) {
        ml0[y] = live[y] && i < n ? a.ml[at(y, i)] : make_float2(-__builtin_inff(), 0.f);
        part0[y] = live[y] && part < n ? *reinterpret_cast<const vec_t *>(a.part + at(y, part) * HD + i * E) : (vec_t)(0.f);
    }
#pragma unroll
    for (int y = 0; y < Y; ++y) top[y] = ml0[y].x;
    for (int s = i + 32; s < n; s += 32)
#pragma unroll
        for (int y = 0; y < Y; ++y)
            if (live[y]) top[y] = fmaxf(top[y], a.ml[at(y, s)].x);
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
        for (int d = 16; d; d >>= 1) top[y] = fmaxf(top[y], __shfl_xor(top[y], d));
    for (int s0 = 0; s0 < n; s0 += 32) {
        float w[Y];
#pragma unroll
        for (int y = 0; y < Y; ++y) {
            const float2 ml = s0 == 0 ? ml0[y] : live[y] && s0 + i < n ? a.ml[at(y, s0 + i)] : make_float2(-__builtin_inff(), 0.f);
            w[y] = weight_of(ml.x, top[y]);
            l[y] += w[y] * ml.y;
        }
        const int nb = min(32, n - s0);
        for (int s1 = 0; s1 < nb; s1 += share) {
            const int s = s1 + part;
#pragma unroll
            for (int y = 0; y < Y; ++y) {
                const float ws = __shfl(w[y], (lane & 32) + (s & 31));
                if (live[y] && s < nb)
                    acc[y] += ws * (s0 + s1 == 0 ? part0[y] : *reinterpret_cast<const vec_t *>(a.part + at(y, s0 + s) * HD + i * E));
            }
        }
    }
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
        for (int d = 16; d; d >>= 1) l[y] += __shfl_xor(l[y], d);
    if (share > 1) {   // 8 rows at most: a half wave has one of them
        s_acc[half][i] = acc[0];
        __syncthreads();
        if (part == 0)
            for (int w = 1; w < share; ++w) acc[0] += s_acc[half + w][i];
    }
#pragma unroll
    for (int y = 0; y < Y; ++y) {
        if (!live[y] || part != 0) continue;
        const vec_t v = acc[y] * inverse_of(l[y]);
        uint16_t *to = a.O + o_at[y] + i * E;
        if constexpr (E == 4) *reinterpret_cast<u32x2_t *>(to) = (u32x2_t){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else *reinterpret_cast<uint32_t *>(to) = pack_bf16x2(v[0], v[1]);
    }
}

inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Waves that group the candidates: their counts, one per wave and user, stay within 128 KB of LDS.
inline int prep_waves(int B_u) { return std::max(1, std::min(kPrep / 64, 32768 / B_u)); }

template <int HD>
hipError_t launch(const AttnArgs &a, int64_t line_most, hipStream_t s) {
    hipError_t e = hipSuccess;
    const bool wide = a.R == 256, small = !wide && a.B_u <= kSmallUsers && a.B_c <= kSmallCands;
    if (!small) {
        const int waves = a.map ? prep_waves(a.B_u) : 0;
        const size_t lds = ((size_t)waves * a.B_u + a.B_u + 1) * sizeof(int);
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kv4_prep_kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 152 * 1024);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kv4_prep_kernel, dim3(1), dim3(kPrep), lds, s, a, waves);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    // No more blocks than pages; a block past the line's end returns at once.
    const dim3 grid((unsigned)std::min<int64_t>(line_most, 1ll << a.log_blocks));
    if (wide) {
        const auto k = kv4_wide_kernel<HD>;
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, kBuffers * WideLds<HD>::PAGE);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k, grid, dim3(512), kBuffers * WideLds<HD>::PAGE, s, a);
    } else {
        // With 16 rows to a unit hardly any two units share a tile, and a cache larger than the 256 MB of the last level
        // is read past it: 97 -> 87 us for 0.46 GB; 0.1 GB, which stays there from call to call, would take 35 for 34.  The
        // table's capacity stands for the cache's size: a wide table over few pages is read past the caches too.
        const bool once = a.R == 16 && (int64_t)a.B_u * a.max_pages * a.H_kv * (68 * HD) > (256ll << 20);
        const auto k = a.R != 16 ? (small ? kv4_attn_kernel<HD, 2, true, false> : kv4_attn_kernel<HD, 2, false, false>)
                       : once    ? (small ? kv4_attn_kernel<HD, 1, true, true> : kv4_attn_kernel<HD, 1, false, true>)
                                 : (small ? kv4_attn_kernel<HD, 1, true, false> : kv4_attn_kernel<HD, 1, false, false>);
        hipLaunchKernelGGL(k, grid, dim3(64), 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.max_pages > 1) {   // a history of one page is never cut
        if (wide) hipLaunchKernelGGL((kv4_join_kernel<HD, 2>), dim3(grid.x, (unsigned)(a.R / 32)), dim3(512), 0, s, a);
        else hipLaunchKernelGGL((kv4_join_kernel<HD, 1>), dim3(grid.x, (unsigned)(a.R / 16)), dim3(512), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

Kv4AttnLayout kv4_attn_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages) {
    Kv4AttnLayout w{};
    const int64_t rows = (int64_t)B_c * L_q * (H_q / H_kv);
    // By the rows of the average user.  32 users of 3000 tokens and 8 heads, in us, narrow against wide: head 128:
    // 106, 143, 181, 320 against 138, 145, 158, 273 at 128, 192, 256, 512 rows; head 64: 80, 104, 129, 220 against
    // 99, 106, 112, 189.  Units of 16 rows against 32: head 128: 36, 43, 50 against 46, 48, 56 at 16, 17, 32 rows, head
    // 64: 31, 39, 45 against 33, 34, 41: between 17 and 32 rows head 128 would rather keep 16.
    // A user is a row of the table, with candidates or without, for the host does not see the map.  15 users with 4352
    // rows each take 159 us in a table of their own, 178 in one of 400 (units of 32 rows) and 334 in one of 4096 (of 16);
    // with one token each 12, 22 and 28 us, most of it the launch that forms the plan.
    const int64_t mean = rows / B_u;
    w.R = mean <= 16 ? 16 : mean <= 192 ? 32 : 256;
    w.log_blocks = w.R == 256 ? kLogWide : kLogNarrow;
    const int64_t tiles = (rows / w.R + std::min(B_u, B_c)) * H_kv;   // at most
    w.line_most = std::max<int64_t>(1, tiles * max_pages);
    const int64_t blocks = std::min<int64_t>(w.line_most, 1ll << w.log_blocks), slots = max_pages > 1 ? 2 * blocks : 0;
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t o = at; at = up(at + bytes, 256); return o; };
    w.o_share = take(8);
    w.o_work = take((int64_t)(B_u + 1) * 8);
    w.o_perm = take((int64_t)B_c * 4);
    w.o_off = take((int64_t)(B_u + 1) * 4);
    w.o_note = take(blocks * 8);
    w.o_note_o = take(blocks * w.R * 8);
    w.o_ml = take(slots * w.R * 8);
    w.o_part = take(slots * w.R * head_dim * 4);
    w.total = at;
    return w;
}

hipError_t launch_kv4_attention(const ikbo_kv4_attention_args &x, const Kv4AttnLayout &w, float scale, hipStream_t s) {
    AttnArgs a{};
    char *ws = static_cast<char *>(x.workspace);
    a.Q = static_cast<const uint16_t *>(x.Q);
    a.O = static_cast<uint16_t *>(x.O);
    a.tiles = static_cast<const char *>(x.tiles);
    a.table = x.block_table; a.lens = x.lens; a.map = x.map; a.positions = x.positions; a.status = x.status;
    a.share = reinterpret_cast<int64_t *>(ws + w.o_share);
    a.work = reinterpret_cast<int64_t *>(ws + w.o_work);
    a.perm = reinterpret_cast<int32_t *>(ws + w.o_perm);
    a.off = reinterpret_cast<int32_t *>(ws + w.o_off);
    a.note = reinterpret_cast<int2 *>(ws + w.o_note);
    a.note_o = reinterpret_cast<int64_t *>(ws + w.o_note_o);
    a.ml = reinterpret_cast<float2 *>(ws + w.o_ml);
    a.part = reinterpret_cast<float *>(ws + w.o_part);
    a.q_cand = x.q_cand; a.q_head = x.q_head; a.q_query = x.q_query;
    a.o_cand = x.o_cand; a.o_head = x.o_head; a.o_query = x.o_query;
    a.table_stride = x.table_stride;
    a.B_u = x.B_u; a.B_c = x.B_c; a.H_kv = x.H_kv; a.G = x.H_q / x.H_kv; a.L_q = x.L_q;
    a.max_pages = x.max_pages; a.num_pages = x.num_pages;
    a.R = w.R; a.log_blocks = w.log_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    return x.head_dim == 128 ? launch<128>(a, w.line_most, s) : launch<64>(a, w.line_most, s);
}

}  // namespace ikbo
