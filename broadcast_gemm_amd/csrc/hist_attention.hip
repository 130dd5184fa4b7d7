// hist_attention.hip -- target attention over the 4-bit paged cache (ikbo_kv4_attention).
//
// For one user and one key/value head, every query row of the user's candidates (candidate, query,
// head of the group) multiplies the same cached K and V: the rows stand beside one another in the
// matrix operands, 16 to a tile, and the cache is read once for all of them, never per candidate.
//
// Per page of 64 tokens a wave forms S^T = K Q^T and O^T += V^T P^T with v_mfma_f32_16x16x32_bf16.
// Codes go from memory to registers and through the hardware's 4-bit conversion (which applies the
// block's scale) straight into operand registers; nothing passes through LDS.  With lane = 16 g + j:
//   S^T tile t (A: keys, B: queries): row j of the tile is token 16 (j / 4) + 4 t + j % 4, so lane
//   (g, j) ends up with query j against tokens 16 g + 4 t + i, i < 4: over the four tiles 16
//   consecutive tokens, 16 g .. 16 g + 15.  Those are the k slots that it must supply as B operand
//   P^T, and the tokens of its A operand V^T: 16 consecutive bytes of a row of the tile's V codes.
//   The d order of the S^T product is free as long as K and Q agree: lane group g takes the g-th
//   quarter of a head, a 16- or 8-byte piece of a K row.
//   A byte of V codes holds elements 2c, 2c + 1 of one token: the low halves of the converted pairs
//   are the operand of the even elements' O^T tile, the high halves that of the odd ones'.
// The running maximum is kept per query; it moves (and O^T is rescaled) only when a page's maximum
// exceeds it by more than 8 (in base 2), so weights stay below 2^8.
//
// Work split: a unit is (user, head, row tile, range of pages).  A grouping launch sorts the
// candidates by user and cuts the histories into about as many units as the chip holds at once
// (twice as many blocks in the wide kernel), whatever the lengths; a unit that covers all pages of
// its rows stores O, the others leave float32 partial results and their maxima and sums, which a
// last launch joins.
//
// Two kernels.  Up to 32 rows per user and head on average, a unit is one wave, which converts the
// codes it reads for itself: the cache's bytes are what counts.  With more rows the conversion would
// be repeated by every wave: a block of 4 waves, 32 rows each, converts a page once into LDS (bf16,
// two pages deep) and each wave reads its operands there.
#include "hist_internal.h"

#include <algorithm>

#include "lce_device.h"

namespace ikbo {
namespace {

constexpr int kPage = IKBO_KV4_PAGE;
constexpr int kPrep = 1024;           // threads of the grouping block
constexpr int kNarrowUnits = 4096;    // units aimed at: 16 waves for each of 256 CUs
constexpr int kWideUnits = 1024;      // blocks of 4 waves, two at a time on each CU
constexpr int kWideWaves = 4, kWideRows = 32 * kWideWaves;
constexpr int kPer = IKBO_KV_MAX_USERS / kPrep;   // users per thread of the grouping block
constexpr float kSlack = 8.0f;

struct AttnArgs {
    const uint16_t *Q;
    uint16_t *O;
    const char *tiles;
    const int32_t *table, *lens, *map, *positions;
    uint32_t *status;
    int32_t *hdr, *perm, *off, *ubase, *pbase, *tbase;
    float2 *ml;
    float *part;
    int64_t q_cand, q_head, q_query, o_cand, o_head, o_query, table_stride;
    int B_u, B_c, H_kv, G, L_q, max_pages, num_pages;
    int rows_per_unit, units;         // rows and number of units aimed at
    float scale_log2;
};

// Pieces that a history of `pages` is cut into for about `chunk` pages each (hdr[0]): at most 1.5 chunk.
// Piece s is pages [cut(s), cut(s + 1)).
__device__ __forceinline__ int pieces(int pages, int chunk) { return max(1, (int)((2u * pages + chunk) / (2u * chunk))); }
__device__ __forceinline__ int cut(int pages, int n, int s) { return (int)((int64_t)pages * s / n); }

__device__ __forceinline__ int clamp_len(int len, int max_pages) { return min(max(len, 0), max_pages * kPage); }

// One block.  Groups the candidates by user (perm, off: a stable counting sort, one run of
// candidates per wave), then the prefix sums over the users of units (ubase), of units that leave
// partial results (pbase) and of row tiles that those join (tbase).
__global__ void __launch_bounds__(kPrep) kv4_prep_kernel(AttnArgs a, int waves) {
    extern __shared__ int sh[];       // counts [waves][B_u], offsets [B_u + 1]
    __shared__ long long s_w[kPrep / 64];
    __shared__ int s_scan[3][kPrep / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int B = a.B_u;
    int *cnt = sh, *offs = sh + waves * B;
    uint32_t err = 0;
    const int per = (B + kPrep - 1) / kPrep;   // consecutive users per thread
    int len_in[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) len_in[e] = e < per && tid * per + e < B ? a.lens[tid * per + e] : 0;

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
        int sum = 0;
        for (int e = 0; e < per; ++e) {
            const int u = tid * per + e;
            if (u < B) {
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
        int inc = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 63) s_scan[0][wv] = inc;
        __syncthreads();
        int base = inc - sum;
        for (int w = 0; w < wv; ++w) base += s_scan[0][w];
        for (int e = 0; e < per; ++e) {
            const int u = tid * per + e;
            if (u < B) {
                const int c = offs[u];
                offs[u] = base;
                base += c;
                if (u == B - 1) offs[B] = base;
            }
        }
        __syncthreads();
        walk([&](int b, int u, bool mine, uint64_t m) {
            int at = 0;
            if (lane == 0) {
                at = cnt[wv * B + u];
                cnt[wv * B + u] = at + __popcll(m);
            }
            at = __shfl(at, 0);
            if (mine) a.perm[offs[u] + at + __popcll(m & ((1ull << lane) - 1))] = b;
        });
        for (int u = tid; u <= B; u += kPrep) a.off[u] = offs[u];
    } else {
        for (int b = tid; b < a.B_c; b += kPrep) a.perm[b] = b;
        for (int u = tid; u <= B; u += kPrep) a.off[u] = offs[u] = min(u, a.B_c);
    }
    __syncthreads();

    // Row tiles and pages of this thread's users, then the pages per unit.
    int tiles[kPer], pages[kPer];
    long long work = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        const bool mine = e < per && u < B;
        const long long rows = mine ? (long long)(offs[u + 1] - offs[u]) * a.L_q * a.G : 0;
        tiles[e] = (int)((rows + a.rows_per_unit - 1) / a.rows_per_unit);
        if (mine && (len_in[e] < 0 || len_in[e] > a.max_pages * kPage)) err |= kStPage;
        pages[e] = (clamp_len(len_in[e], a.max_pages) + kPage - 1) / kPage;
        work += (long long)tiles[e] * pages[e] * a.H_kv;
    }
    for (int d = 32; d; d >>= 1) work += __shfl_xor(work, d);
    if (lane == 0) s_w[wv] = work;
    __syncthreads();
    work = 0;
    for (int w = 0; w < kPrep / 64; ++w) work += s_w[w];
    const int chunk = (int)min(max(1ll, (work + a.units - 1) / a.units), 1ll << 28);

    int v[3] = {0, 0, 0}, inc[3];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int n = pieces(pages[e], chunk);
        v[0] += tiles[e] * n;
        if (n > 1) { v[1] += tiles[e] * n; v[2] += tiles[e]; }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        inc[k] = v[k];
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc[k], d);
            if (lane >= d) inc[k] += o;
        }
        if (lane == 63) s_scan[k][wv] = inc[k];
    }
    __syncthreads();
    int base[3], *const out[3] = {a.ubase, a.pbase, a.tbase};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        base[k] = inc[k] - v[k];
        for (int w = 0; w < wv; ++w) base[k] += s_scan[k][w];
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int u = tid * per + e;
        if (e < per && u < B) {
            const int n = pieces(pages[e], chunk);
#pragma unroll
            for (int k = 0; k < 3; ++k) out[k][u] = base[k];
            base[0] += tiles[e] * n;
            if (n > 1) { base[1] += tiles[e] * n; base[2] += tiles[e]; }
            if (u == B - 1)
#pragma unroll
                for (int k = 0; k < 3; ++k) out[k][B] = base[k];
        }
    }
    if (tid == 0) a.hdr[0] = chunk;
    if (err) atomicOr(a.status, err);
}

// Largest u in [0, n) with base[u] <= x: the owner of x (users without units share their
// successor's base and are skipped).
__device__ __forceinline__ int owner_of(const int32_t *base, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// x against the lanes 16 and 32 away.
__device__ __forceinline__ float max_over_groups(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const float y = fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
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

// The 8 values of one dword of codes.
__device__ __forceinline__ u32x4_t values8(uint32_t codes, float scale) {
    return (u32x4_t){values2<0>(codes, scale), values2<1>(codes, scale), values2<2>(codes, scale), values2<3>(codes, scale)};
}

// What a lane reads of a page.
template <int HD>
struct PageRegs {
    static constexpr int KW = HD / 32;     // dwords of a K row per lane
    static constexpr int VJ = HD / 32;     // 16-pair groups of V rows
    uint32_t k[4][KW];
    uint32_t ks;
    u32x4_t v[VJ], vs[VJ];
    __device__ __forceinline__ void load_k(const char *tile, int g, int j) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const char *p = tile + (16 * (j >> 2) + 4 * t + (j & 3)) * (HD / 2) + g * (HD / 8);
            if constexpr (HD == 128) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) k[t][i] = w[i];
            } else {
                const u32x2_t w = *reinterpret_cast<const u32x2_t *>(p);
                k[t][0] = w[0];
                k[t][1] = w[1];
            }
        }
        ks = *reinterpret_cast<const uint32_t *>(tile + 64 * HD + (HD == 128 ? g : g >> 1) * 64 + 4 * j);
    }
    __device__ __forceinline__ void load_v(const char *tile, int g, int j) {
#pragma unroll
        for (int jj = 0; jj < VJ; ++jj) {
            v[jj] = *reinterpret_cast<const u32x4_t *>(tile + 32 * HD + (16 * jj + j) * 64 + 16 * g);
            vs[jj] = *reinterpret_cast<const u32x4_t *>(tile + 66 * HD + jj * 64 + 16 * g);
        }
    }
};

template <int HD, int NT>
__global__ void __launch_bounds__(64) kv4_attn_kernel(AttnArgs a) {
    constexpr int KS = HD / 32;   // 32-wide steps of d
    constexpr int VJ = HD / 32;
    constexpr int TILE = 68 * HD;
    const int lane = (int)threadIdx.x, g = lane >> 4, j = lane & 15;
    const int chunk = a.hdr[0], n_units = a.ubase[a.B_u] * a.H_kv;
    for (int unit = (int)blockIdx.x; unit < n_units; unit += (int)gridDim.x) {
        // Units of a user in the order split, head, row tile: neighbours share their K and V.
        const int u = owner_of(a.ubase, a.B_u, unit / a.H_kv);
        const int c0 = a.off[u], n_rows = (a.off[u + 1] - c0) * a.L_q * a.G;
        const int tiles = (n_rows + 16 * NT - 1) / (16 * NT);
        const int local = unit - a.ubase[u] * a.H_kv;
        const int tile_i = local % tiles, h = local / tiles % a.H_kv, split = local / tiles / a.H_kv;
        const int len = clamp_len(a.lens[u], a.max_pages);
        const int pages = (len + kPage - 1) / kPage;
        const int n_pieces = pieces(pages, chunk);
        const bool whole = n_pieces == 1;
        const int p0 = cut(pages, n_pieces, split);

        // This lane's query rows j, 16 + j, ..: their candidate, query and head, and what they see.
        int64_t o_at[NT];
        int limit[NT];
        u32x4_t qf[KS][NT];
        bool live[NT];
        int most = 0, least = len;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = tile_i * 16 * NT + 16 * n + j;
            live[n] = row < n_rows;
            const int r = live[n] ? row : 0;
            const int cand = a.perm[c0 + r / (a.L_q * a.G)], rest = r % (a.L_q * a.G);
            const int l = rest / a.G, hq = h * a.G + rest % a.G;
            o_at[n] = cand * a.o_cand + hq * a.o_head + l * a.o_query;
            limit[n] = live[n] ? len : 0;
            if (live[n] && a.positions) {
                const int pos = a.positions[(int64_t)cand * a.L_q + l];
                limit[n] = pos < 0 ? 0 : pos < len ? pos + 1 : len;
            }
            const uint16_t *q = a.Q + cand * a.q_cand + hq * a.q_head + l * a.q_query + g * (HD / 4);
#pragma unroll
            for (int s = 0; s < KS; ++s)
                qf[s][n] = live[n] ? *reinterpret_cast<const u32x4_t *>(q + 8 * s) : (u32x4_t){0, 0, 0, 0};
            most = max(most, limit[n]);
            if (live[n]) least = min(least, limit[n]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            most = max(most, __shfl_xor(most, d));
            least = min(least, __shfl_xor(least, d));
        }
        most = __builtin_amdgcn_readfirstlane(most);
        least = __builtin_amdgcn_readfirstlane(least);
        const int p1 = min(cut(pages, n_pieces, split + 1), (most + kPage - 1) / kPage);   // no row sees further pages

        f32x4_t o[2 * VJ][NT], lsum[NT];
        float m[NT], nm[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -__builtin_inff();
            nm[n] = 0.f;
            lsum[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 2 * VJ; ++x) o[x][n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        }
        const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const int32_t *row = a.table + (int64_t)u * a.table_stride;
        bool bad_page = false;
        auto tile_at = [&](int p) {
            int page = __builtin_amdgcn_readfirstlane(row[p]);
            if (page < 0 || page >= a.num_pages) { bad_page = true; page = 0; }
            return a.tiles + ((int64_t)page * a.H_kv + h) * TILE;
        };
        PageRegs<HD> pg;
        for (int p = p0; p < p1; ++p) {
            const char *tile = tile_at(p);
            pg.load_k(tile, g, j);
            pg.load_v(tile, g, j);
            f32x4_t S[4][NT];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float ks = scale_of(pg.ks, t);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[t][n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const u32x4_t kf = values8(pg.k[t][s], ks);
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[t][n] = mfma_bf16(kf, qf[s][n], S[t][n]);
                }
            }
            const int key0 = p * kPage + 16 * g;   // this lane's tokens: key0 + 4 t + i
            if (p * kPage + kPage > least) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (key0 + 4 * t + i >= limit[n]) S[t][n][i] = -__builtin_inff();
            }
            if (p * kPage + kPage > len) {
                // Tokens past the history may hold anything: scale 2^-127 keeps their values finite,
                // and their weights are 0.
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int n = len - (key0 + 4 * t);
                    const uint32_t keep = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
#pragma unroll
                    for (int jj = 0; jj < VJ; ++jj) pg.vs[jj][t] &= keep;
                }
            }
            bool grow = false;
            float mb[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x = -__builtin_inff();
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x = fmaxf(x, S[t][n][i]);
                mb[n] = max_over_groups(x) * a.scale_log2;
                grow = grow || mb[n] > m[n] + kSlack;
            }
            if (__ballot(grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float mn = fmaxf(m[n], mb[n]);
                    const float alpha = mn == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                    m[n] = mn;
                    nm[n] = mn == -__builtin_inff() ? 0.f : -mn;
                    lsum[n] *= alpha;
#pragma unroll
                    for (int x = 0; x < 2 * VJ; ++x) o[x][n] *= alpha;
                }
            }
            u32x4_t pf[2][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[t][n][i], a.scale_log2, nm[n]));
                    pf[t >> 1][n][2 * (t & 1)] = pack_bf16x2(w[0], w[1]);
                    pf[t >> 1][n][2 * (t & 1) + 1] = pack_bf16x2(w[2], w[3]);
                }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int n = 0; n < NT; ++n) lsum[n] = mfma_bf16(ones, pf[kk][n], lsum[n]);
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    u32x4_t even, odd;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t c = pg.v[jj][2 * kk + x], s = pg.vs[jj][2 * kk + x];
                        const uint32_t v0 = values2<0>(c, scale_of(s, 0)), v1 = values2<1>(c, scale_of(s, 1));
                        const uint32_t v2 = values2<2>(c, scale_of(s, 2)), v3 = values2<3>(c, scale_of(s, 3));
                        even[2 * x] = pair16(v0, v1, false);
                        even[2 * x + 1] = pair16(v2, v3, false);
                        odd[2 * x] = pair16(v0, v1, true);
                        odd[2 * x + 1] = pair16(v2, v3, true);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[2 * jj][n] = mfma_bf16(even, pf[kk][n], o[2 * jj][n]);
                        o[2 * jj + 1][n] = mfma_bf16(odd, pf[kk][n], o[2 * jj + 1][n]);
                    }
                }
            }
        }
        if (bad_page && lane == 0) atomicOr(a.status, kStPage);

        // Lane (g, j) holds of query j the elements 32 jj + 8 g + 2 i (even tile) and + 1 (odd tile).
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (!live[n]) continue;
            const float l = lsum[n][0];
            if (whole) {
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;   // a row that sees nothing is 0
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    u32x4_t w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(o[2 * jj][n][i] * inv, o[2 * jj + 1][n][i] * inv);
                    *reinterpret_cast<u32x4_t *>(a.O + o_at[n] + 32 * jj + 8 * g) = w;
                }
            } else {
                // Partial results in the units' order.
                const int64_t at = ((int64_t)(unit - (a.ubase[u] - a.pbase[u]) * a.H_kv)) * (16 * NT) + 16 * n + j;
                if (g == 0) a.ml[at] = make_float2(m[n], l);
                float *to = a.part + at * HD;
#pragma unroll
                for (int jj = 0; jj < VJ; ++jj) {
                    f32x4_t w0, w1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        w0[2 * i] = o[2 * jj][n][i];
                        w0[2 * i + 1] = o[2 * jj + 1][n][i];
                        w1[2 * i] = o[2 * jj][n][2 + i];
                        w1[2 * i + 1] = o[2 * jj + 1][n][2 + i];
                    }
                    *reinterpret_cast<f32x4_t *>(to + 32 * jj + 8 * g) = w0;
                    *reinterpret_cast<f32x4_t *>(to + 32 * jj + 8 * g + 4) = w1;
                }
            }
        }
    }
}

// ---- the wide kernel -----------------------------------------------------------------------

// A page in LDS: K rows [64 tokens][HD] and V^T rows [HD][64 tokens], bf16.  The 16-byte chunks of a
// row stand permuted by an XOR with a row number so that the 16 rows of one operand read fall on
// different banks: for K the row's place j in the operand, for V^T the row itself.
template <int HD>
struct WideLds {
    static constexpr int KBYTES = kPage * HD * 2, PAGE = 2 * KBYTES;
    static __device__ __forceinline__ int k_at(int key, int c) {
        const int j = 4 * (key >> 4) + (key & 3);
        return key * HD * 2 + ((c ^ (j & (HD / 8 - 1))) << 4);
    }
    static __device__ __forceinline__ int v_at(int d, int c) { return KBYTES + d * kPage * 2 + ((c ^ (d & 7)) << 4); }
};

template <int HD>
__global__ void __launch_bounds__(64 * kWideWaves, 2) kv4_wide_kernel(AttnArgs a) {
    typedef WideLds<HD> L;
    constexpr int NT = 2, TK = HD / 32, DT = HD / 16, TILE = 68 * HD;
    constexpr int JOBS = kPage * HD / 16 / (64 * kWideWaves);   // 8-byte pieces of K codes (and of V codes) per thread
    extern __shared__ __align__(16) char lds[];
    __shared__ int s_most[kWideWaves];
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6, g = lane >> 4, j = lane & 15;
    const int chunk = a.hdr[0], n_units = a.ubase[a.B_u] * a.H_kv;
    for (int unit = (int)blockIdx.x; unit < n_units; unit += (int)gridDim.x) {
        const int u = owner_of(a.ubase, a.B_u, unit / a.H_kv);
        const int c0 = a.off[u], n_rows = (a.off[u + 1] - c0) * a.L_q * a.G;
        const int tiles = (n_rows + kWideRows - 1) / kWideRows;
        const int local = unit - a.ubase[u] * a.H_kv;
        const int tile_i = local % tiles, h = local / tiles % a.H_kv, split = local / tiles / a.H_kv;
        const int len = clamp_len(a.lens[u], a.max_pages);
        const int pages = (len + kPage - 1) / kPage;
        const int n_pieces = pieces(pages, chunk);
        const bool whole = n_pieces == 1;
        const int p0 = cut(pages, n_pieces, split);

        int64_t o_at[NT];
        int limit[NT];
        u32x4_t qf[TK][NT];
        bool live[NT];
        int most = 0, least = len;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = tile_i * kWideRows + wv * 16 * NT + 16 * n + j;
            live[n] = row < n_rows;
            const int r = live[n] ? row : 0;
            const int cand = a.perm[c0 + r / (a.L_q * a.G)], rest = r % (a.L_q * a.G);
            const int l = rest / a.G, hq = h * a.G + rest % a.G;
            o_at[n] = cand * a.o_cand + hq * a.o_head + l * a.o_query;
            limit[n] = live[n] ? len : 0;
            if (live[n] && a.positions) {
                const int pos = a.positions[(int64_t)cand * a.L_q + l];
                limit[n] = pos < 0 ? 0 : pos < len ? pos + 1 : len;
            }
            const uint16_t *q = a.Q + cand * a.q_cand + hq * a.q_head + l * a.q_query + 8 * g;
#pragma unroll
            for (int t = 0; t < TK; ++t)
                qf[t][n] = live[n] ? *reinterpret_cast<const u32x4_t *>(q + 32 * t) : (u32x4_t){0, 0, 0, 0};
            most = max(most, limit[n]);
            if (live[n]) least = min(least, limit[n]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            most = max(most, __shfl_xor(most, d));
            least = min(least, __shfl_xor(least, d));
        }
        most = __builtin_amdgcn_readfirstlane(most);
        least = __builtin_amdgcn_readfirstlane(least);
        if (lane == 0) s_most[wv] = most;
        __syncthreads();   // also: the block's last reads of the previous unit's pages are done
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWideWaves; ++w) all = max(all, s_most[w]);
        const int p1 = min(cut(pages, n_pieces, split + 1), (all + kPage - 1) / kPage);   // no row sees further pages

        f32x4_t o[DT][NT], lsum[NT];
        float m[NT], nm[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -__builtin_inff();
            nm[n] = 0.f;
            lsum[n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < DT; ++x) o[x][n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
        }
        const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const int32_t *row = a.table + (int64_t)u * a.table_stride;
        bool bad_page = false;

        // Codes and scales of a page, this thread's pieces: K piece c is 16 elements of token
        // c / (HD/16); V piece c is 8 tokens of element pair c / 8.
        u32x2_t kc[JOBS], vc[JOBS], vs[JOBS];
        uint32_t ks[JOBS];
        auto fetch = [&](int p) {
            int page = __builtin_amdgcn_readfirstlane(row[p]);
            if (page < 0 || page >= a.num_pages) { bad_page = true; page = 0; }
            const char *tile = a.tiles + ((int64_t)page * a.H_kv + h) * TILE;
#pragma unroll
            for (int i = 0; i < JOBS; ++i) {
                const int c = tid + i * 64 * kWideWaves;
                const int key = c / (HD / 16), part = c % (HD / 16);
                kc[i] = *reinterpret_cast<const u32x2_t *>(tile + 8 * c);
                ks[i] = (uint8_t)tile[64 * HD + (part >> 1) * 64 + (key & 48) + 4 * (key & 3) + ((key >> 2) & 3)];
                vc[i] = *reinterpret_cast<const u32x2_t *>(tile + 32 * HD + 8 * c);
                vs[i] = *reinterpret_cast<const u32x2_t *>(tile + 66 * HD + (c >> 7) * 64 + 8 * (c & 7));
            }
        };
        auto convert = [&](int p) {
            char *to = lds + (p & 1) * L::PAGE;
#pragma unroll
            for (int i = 0; i < JOBS; ++i) {
                const int c = tid + i * 64 * kWideWaves;
                const int key = c / (HD / 16), part = c % (HD / 16);
                const float s = scale_of(ks[i], 0);
                *reinterpret_cast<u32x4_t *>(to + L::k_at(key, 2 * part)) = values8(kc[i][0], s);
                *reinterpret_cast<u32x4_t *>(to + L::k_at(key, 2 * part + 1)) = values8(kc[i][1], s);
                const int pair = c >> 3, k0 = 8 * (c & 7);
                u32x4_t even, odd;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t sc = vs[i][x];
                    // Tokens past the history may hold anything: scale 2^-127 keeps their values
                    // finite, and their weights are 0.
                    const int n = len - (p * kPage + k0 + 4 * x);
                    if (n < 4) sc &= n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    const uint32_t v0 = values2<0>(vc[i][x], scale_of(sc, 0)), v1 = values2<1>(vc[i][x], scale_of(sc, 1));
                    const uint32_t v2 = values2<2>(vc[i][x], scale_of(sc, 2)), v3 = values2<3>(vc[i][x], scale_of(sc, 3));
                    even[2 * x] = pair16(v0, v1, false);
                    even[2 * x + 1] = pair16(v2, v3, false);
                    odd[2 * x] = pair16(v0, v1, true);
                    odd[2 * x + 1] = pair16(v2, v3, true);
                }
                *reinterpret_cast<u32x4_t *>(to + L::v_at(2 * pair, k0 >> 3)) = even;
                *reinterpret_cast<u32x4_t *>(to + L::v_at(2 * pair + 1, k0 >> 3)) = odd;
            }
        };
        if (p0 < p1) {
            fetch(p0);
            convert(p0);
            if (p0 + 1 < p1) fetch(p0 + 1);
        }
        __syncthreads();
        for (int p = p0; p < p1; ++p) {
            const char *from = lds + (p & 1) * L::PAGE;
            f32x4_t S[4][NT];
            const bool busy = p * kPage < most;   // some row of this wave sees the page
            if (busy) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[t][n] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < TK; ++s)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const u32x4_t kf = *reinterpret_cast<const u32x4_t *>(from + L::k_at(16 * (j >> 2) + 4 * t + (j & 3), 4 * s + g));
#pragma unroll
                        for (int n = 0; n < NT; ++n) S[t][n] = mfma_bf16(kf, qf[s][n], S[t][n]);
                    }
            }
            // The other page buffer was last read before the barrier that ended the previous turn.
            if (p + 1 < p1) {
                convert(p + 1);
                if (p + 2 < p1) fetch(p + 2);
            }
            if (busy) {
                const int key0 = p * kPage + 16 * g;   // this lane's tokens: key0 + 4 t + i
                if (p * kPage + kPage > least) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (key0 + 4 * t + i >= limit[n]) S[t][n][i] = -__builtin_inff();
                }
                bool grow = false;
                float mb[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x = -__builtin_inff();
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x = fmaxf(x, S[t][n][i]);
                    mb[n] = max_over_groups(x) * a.scale_log2;
                    grow = grow || mb[n] > m[n] + kSlack;
                }
                if (__ballot(grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float mn = fmaxf(m[n], mb[n]);
                        const float alpha = mn == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                        m[n] = mn;
                        nm[n] = mn == -__builtin_inff() ? 0.f : -mn;
                        lsum[n] *= alpha;
#pragma unroll
                        for (int x = 0; x < DT; ++x) o[x][n] *= alpha;
                    }
                }
                u32x4_t pf[2][NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[t][n][i], a.scale_log2, nm[n]));
                        pf[t >> 1][n][2 * (t & 1)] = pack_bf16x2(w[0], w[1]);
                        pf[t >> 1][n][2 * (t & 1) + 1] = pack_bf16x2(w[2], w[3]);
                    }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) lsum[n] = mfma_bf16(ones, pf[kk][n], lsum[n]);
#pragma unroll
                    for (int x = 0; x < DT; ++x) {
                        const u32x4_t vf = *reinterpret_cast<const u32x4_t *>(from + L::v_at(16 * x + j, 2 * g + kk));
#pragma unroll
                        for (int n = 0; n < NT; ++n) o[x][n] = mfma_bf16(vf, pf[kk][n], o[x][n]);
                    }
                }
            }
            __syncthreads();
        }
        if (bad_page && tid == 0) atomicOr(a.status, kStPage);

        // Lane (g, j) holds of query j the elements 16 x + 4 g + i.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (!live[n]) continue;
            const float l = lsum[n][0];
            if (whole) {
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;   // a row that sees nothing is 0
#pragma unroll
                for (int x = 0; x < DT; ++x)
                    *reinterpret_cast<u32x2_t *>(a.O + o_at[n] + 16 * x + 4 * g) =
                        (u32x2_t){pack_bf16x2(o[x][n][0] * inv, o[x][n][1] * inv), pack_bf16x2(o[x][n][2] * inv, o[x][n][3] * inv)};
            } else {
                const int64_t at = ((int64_t)(unit - (a.ubase[u] - a.pbase[u]) * a.H_kv)) * kWideRows + wv * 16 * NT + 16 * n + j;
                if (g == 0) a.ml[at] = make_float2(m[n], l);
#pragma unroll
                for (int x = 0; x < DT; ++x) *reinterpret_cast<f32x4_t *>(a.part + at * HD + 16 * x + 4 * g) = o[x][n];
            }
        }
    }
}

// Joins the partial results of the row tiles that were split: O = sum_s w_s O_s / sum_s w_s l_s with
// w_s = 2^(m_s - max m).  A block per row: the pieces' weights once into LDS, then wave w sums the
// pieces w, w + 4, .. (lane i: HD/64 neighbouring elements), and the four sums meet in LDS.
template <int HD>
__global__ void __launch_bounds__(256) kv4_join_kernel(AttnArgs a) {
    constexpr int E = HD / 64, kBatch = 512;
    __shared__ float s_wt[kBatch], s_sum[4][HD], s_red[4], s_l[4];
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int R = a.rows_per_unit;
    const int64_t n_rows_all = (int64_t)a.tbase[a.B_u] * a.H_kv * R;
    const int chunk = a.hdr[0];
    for (int64_t x = blockIdx.x; x < n_rows_all; x += gridDim.x) {
        const int th = (int)(x / R), r_in = (int)(x % R);
        const int u = owner_of(a.tbase, a.B_u, th / a.H_kv);
        const int c0 = a.off[u], n_rows = (a.off[u + 1] - c0) * a.L_q * a.G;
        const int tiles = (n_rows + R - 1) / R;
        const int local = th - a.tbase[u] * a.H_kv;
        const int tile_i = local % tiles, h = local / tiles;
        const int r = tile_i * R + r_in;
        if (r >= n_rows) continue;
        const int n = pieces((clamp_len(a.lens[u], a.max_pages) + kPage - 1) / kPage, chunk);
        const int64_t first = ((int64_t)a.pbase[u] * a.H_kv + h * tiles + tile_i) * R + r_in;
        const int64_t step = (int64_t)tiles * a.H_kv * R;
        float top = -__builtin_inff();
        for (int s = tid; s < n; s += 256) top = fmaxf(top, a.ml[first + s * step].x);
        for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        if (lane == 0) s_red[wv] = top;
        __syncthreads();
        top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
        float acc[E] = {}, l = 0.f;
        for (int s0 = 0; s0 < n; s0 += kBatch) {
            const int nb = min(kBatch, n - s0);
            for (int s = tid; s < nb; s += 256) {
                const float2 ml = a.ml[first + (s0 + s) * step];
                const float w = ml.x == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
                s_wt[s] = w;
                l += w * ml.y;
            }
            __syncthreads();
            const float *p = a.part + (first + s0 * step) * HD + lane * E;
#pragma unroll 8
            for (int s = wv; s < nb; s += 4) {
                const float w = s_wt[s];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += w * p[s * step * HD + e];
            }
            __syncthreads();
        }
        for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
        if (lane == 0) s_l[wv] = l;
#pragma unroll
        for (int e = 0; e < E; ++e) s_sum[wv][lane * E + e] = acc[e];
        __syncthreads();
        if (tid < HD / 2) {
            l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                y[e] = ((s_sum[0][2 * tid + e] + s_sum[1][2 * tid + e]) + (s_sum[2][2 * tid + e] + s_sum[3][2 * tid + e])) * inv;
            const int cand = a.perm[c0 + r / (a.L_q * a.G)], rest = r % (a.L_q * a.G);
            uint16_t *to = a.O + cand * a.o_cand + (int64_t)(h * a.G + rest % a.G) * a.o_head + (int64_t)(rest / a.G) * a.o_query;
            reinterpret_cast<uint32_t *>(to)[tid] = pack_bf16x2(y[0], y[1]);
        }
        __syncthreads();
    }
}

inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Waves that group the candidates: their counts, one per wave and user, stay within 128 KB of LDS.
inline int prep_waves(int B_u) { return std::max(1, std::min(kPrep / 64, 32768 / B_u)); }

template <int HD>
hipError_t launch(const AttnArgs &a, int64_t max_units, hipStream_t s) {
    const int waves = a.map ? prep_waves(a.B_u) : 0;
    const size_t lds = ((size_t)waves * a.B_u + a.B_u + 1) * sizeof(int);
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kv4_prep_kernel),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, 152 * 1024);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kv4_prep_kernel, dim3(1), dim3(kPrep), lds, s, a, waves);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 grid((unsigned)std::min<int64_t>(max_units, 2 * a.units));
    if (a.rows_per_unit == 16) hipLaunchKernelGGL((kv4_attn_kernel<HD, 1>), grid, dim3(64), 0, s, a);
    else if (a.rows_per_unit == 32) hipLaunchKernelGGL((kv4_attn_kernel<HD, 2>), grid, dim3(64), 0, s, a);
    else {
        const auto k = kv4_wide_kernel<HD>;
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(k), hipFuncAttributeMaxDynamicSharedMemorySize, 2 * WideLds<HD>::PAGE);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k, grid, dim3(64 * kWideWaves), 2 * WideLds<HD>::PAGE, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.max_pages > 1) {   // a history of one page is never split
        const int64_t rows = (int64_t)a.B_c * a.L_q * a.G * a.H_kv;
        hipLaunchKernelGGL(kv4_join_kernel<HD>, dim3((unsigned)std::min<int64_t>(rows, 2048)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

Kv4AttnLayout kv4_attn_layout(int B_u, int B_c, int H_q, int H_kv, int L_q, int head_dim, int max_pages) {
    Kv4AttnLayout w{};
    const int64_t rows = (int64_t)B_c * L_q * (H_q / H_kv);
    // Rows beside one another in a wave: as many tiles of 16 as the average user's rows fill.
    const int64_t mean = rows / B_u;
    w.rows_per_unit = mean <= 16 ? 16 : mean <= 32 ? 32 : kWideRows;
    w.units = w.rows_per_unit <= 32 ? kNarrowUnits : kWideUnits;
    const int64_t tiles = (rows / w.rows_per_unit + std::min(B_u, B_c)) * H_kv;   // at most
    // A history of 1.5 chunk pages or more is cut into at most pages / chunk + 1/2 <= 4/3 pages / chunk
    // pieces, and all pages over the chunk are at most the units aimed at.
    w.part_units = max_pages > 1 ? std::min<int64_t>(2 * w.units, tiles * max_pages) : 0;
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t o = at; at = up(at + bytes, 256); return o; };
    w.o_hdr = take(64);
    w.o_perm = take((int64_t)B_c * 4);
    w.o_off = take((int64_t)(B_u + 1) * 4);
    w.o_ubase = take((int64_t)(B_u + 1) * 4);
    w.o_pbase = take((int64_t)(B_u + 1) * 4);
    w.o_tbase = take((int64_t)(B_u + 1) * 4);
    w.o_ml = take(w.part_units * w.rows_per_unit * 8);
    w.o_part = take(w.part_units * w.rows_per_unit * head_dim * 4);
    w.total = at;
    return w;
}

hipError_t launch_kv4_attention(const ikbo_kv4_attention_args &x, const Kv4AttnLayout &w, float scale, hipStream_t s) {
    AttnArgs a{};
    char *ws = static_cast<char *>(x.workspace);
    auto i32 = [&](int64_t o) { return reinterpret_cast<int32_t *>(ws + o); };
    a.Q = static_cast<const uint16_t *>(x.Q);
    a.O = static_cast<uint16_t *>(x.O);
    a.tiles = static_cast<const char *>(x.tiles);
    a.table = x.block_table; a.lens = x.lens; a.map = x.map; a.positions = x.positions; a.status = x.status;
    a.hdr = i32(w.o_hdr); a.perm = i32(w.o_perm); a.off = i32(w.o_off);
    a.ubase = i32(w.o_ubase); a.pbase = i32(w.o_pbase); a.tbase = i32(w.o_tbase);
    a.ml = reinterpret_cast<float2 *>(ws + w.o_ml);
    a.part = reinterpret_cast<float *>(ws + w.o_part);
    a.q_cand = x.q_cand; a.q_head = x.q_head; a.q_query = x.q_query;
    a.o_cand = x.o_cand; a.o_head = x.o_head; a.o_query = x.o_query;
    a.table_stride = x.table_stride;
    a.B_u = x.B_u; a.B_c = x.B_c; a.H_kv = x.H_kv; a.G = x.H_q / x.H_kv; a.L_q = x.L_q;
    a.max_pages = x.max_pages; a.num_pages = x.num_pages;
    a.rows_per_unit = w.rows_per_unit;
    a.units = w.units;
    a.scale_log2 = scale * 1.4426950408889634f;
    const int64_t rows = (int64_t)x.B_c * x.L_q * a.G;
    const int64_t tiles = (rows / w.rows_per_unit + std::min(x.B_u, x.B_c)) * x.H_kv;
    const int64_t max_units = std::max<int64_t>(1, std::min<int64_t>(tiles * x.max_pages, tiles + w.units));
    return x.head_dim == 128 ? launch<128>(a, max_units, s) : launch<64>(a, max_units, s);
}

}  // namespace ikbo
