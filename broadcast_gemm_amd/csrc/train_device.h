// train_device.h -- what the training kernels of target attention share: operands, staging, random numbers, rows.
//
// All products are v_mfma_f32_32x32x16_bf16; lane = 32 g + j.  A holds row j, contraction 8 g .. + 7; B column j,
// likewise; element i of the result is row 8 (i / 4) + 4 g + i % 4 of column j.  A result that becomes the B operand of
// the next product (weights, or their gradients) is used as it stands: step s of 16 takes elements 8 s .. 8 s + 7, that
// is rows 16 s + 4 g + {0..3} and 16 s + 8 + 4 g + {0..3}, and the A operand of that product holds the same rows of a
// staged matrix, transposed: two ds_read_b64_tr_b16, each 4 rows of column j.
#pragma once

#include "lce_device.h"
#include "lce_sync.h"
#include "train_internal.h"

namespace ikbo {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16_t mfma32(const u32x4_t &a, const u32x4_t &b, f32x16_t acc) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
}

// Nothing is scheduled across.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// x with that of the lane 32 away.
__device__ __forceinline__ float sum_halves(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __builtin_bit_cast(float, (uint32_t)p[0]) + __builtin_bit_cast(float, (uint32_t)p[1]);
}
__device__ __forceinline__ float max_halves(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}

// ---- staged matrices -----------------------------------------------------------------------
//
// Rows of HD bf16 elements in groups of 1 KB (what one load of a wave fills), each row's 16-byte chunks permuted by an
// XOR with a number of the row.  A 16-byte read of a wave is served in sets of 16 lanes that hold each j % 16 once; a
// transposed read takes 64 bytes of each of 4 neighbouring rows.  HD 128: the 4 rows of a group differ in the bits above
// those of 4 chunks, and groups are set off by a chunk, so that the place of step s needs s / 2 alone (fewer registers).  HD 64:
// pairs of rows share 256 bytes, and the number has 3 bits.  Measured without conflicts: 256 bytes a cycle for both reads.
template <int HD>
struct Rows {
    static constexpr int BYTES = HD * 2, CHUNKS = HD / 8, EACH = 1024 / BYTES, GROUP = HD == 128 ? 1040 : 1024;
    static constexpr int matrix(int rows) { return rows / EACH * GROUP; }
    static __device__ __forceinline__ int number(int row) {
        return HD == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int row, int chunk) {
        return row / EACH * GROUP + row % EACH * BYTES + ((chunk ^ number(row)) << 4);
    }
};

// A lane's reads of a staged matrix: row 32 t + j, step s of its elements; and rows 16 s + 4 g + {0..3} (and 8 behind) of
// column 32 d + j.  What depends on t, and on s there, is a constant.
template <int HD>
struct Reader {
    static constexpr int HALF = HD == 128 ? 2 : 1;   // steps that stand side by side whatever the row
    int row[HD / 16 / HALF], col[2 / HALF][HD / 32];
    __device__ __forceinline__ void init(int lane) {
        const int g = lane >> 5, j = lane & 31, i = lane & 15;
#pragma unroll
        for (int s = 0; s < HD / 16 / HALF; ++s) row[s] = Rows<HD>::at(j, 2 * HALF * s + g);
#pragma unroll
        for (int d = 0; d < HD / 32; ++d)
#pragma unroll
            for (int y = 0; y < 2 / HALF; ++y) {   // 16 lanes read 4 rows of 16 columns, 8 bytes each
                const int c = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (i & 3);
                col[y][d] = Rows<HD>::at(8 * y + 4 * g + (i >> 2), c >> 3) + 2 * (c & 7);
            }
    }
    __device__ __forceinline__ u32x4_t direct(const char *m, int t, int s) const {
        return *reinterpret_cast<const u32x4_t *>(m + row[s / HALF] + s % HALF * 32 + Rows<HD>::matrix(32 * t));
    }
    __device__ __forceinline__ u32x4_t turned(const char *m, int s, int d) const {
        u32x2_t w[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
            w[y] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t *)(
                m + col[y / HALF][d] + (HALF == 2 ? Rows<HD>::matrix(8 * y) : 0) + Rows<HD>::matrix(16 * s))));
        return (u32x4_t){w[0][0], w[0][1], w[1][0], w[1][1]};
    }
};

// 16 bytes per lane from device memory straight into LDS, lane l's at `to` + 16 l.  Inline because the compiler would
// make every LDS read wait for the builtin's loads; `landed` waits for them, and a barrier publishes them.  Nothing else in
// these kernels uses m0.
__device__ __forceinline__ void load_to_lds(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory");
}
// The same with a uniform base and an offset per lane.
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) { return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p; }
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// What stands for a row that does not exist.
__device__ const uint32_t kZeroRow[64] __attribute__((aligned(16))) = {};

// A block's staging of 64 keys and their values of one user and head: uniform addresses and one offset per lane, but for the
// last keys of a history.
template <int HD, int WAVES>
struct KeyLoads {
    static constexpr int N = 64 * HD / 8 / (64 * WAVES), STEP = Rows<HD>::EACH * WAVES;   // loads of a matrix, and rows between them
    static_assert(STEP % 16 == 0, "the rows of a lane's loads have one number");
    const char *k, *v;
    int64_t k_row, v_row;   // bytes from token to token
    uint32_t k_off, v_off;
    __device__ __forceinline__ void init(const TrainArgs &a, int u, int hk, int lane, int wv) {
        k = reinterpret_cast<const char *>(a.K + u * a.k_user + hk * a.k_head);
        v = reinterpret_cast<const char *>(a.V + u * a.v_user + hk * a.v_head);
        k_row = 2 * a.k_token;
        v_row = 2 * a.v_token;
        const int row = row_of(wv * 64 + lane), chunk = chunk_of(wv * 64 + lane);
        k_off = (uint32_t)(row * k_row + chunk);   // below 2^32: the host allows tokens 2^24 elements apart
        v_off = (uint32_t)(row * v_row + chunk);
    }
    // Keys t0 .. t0 + 63 (or their values) to `to`; those from `len` on are zeros.
    __device__ __forceinline__ void load_k(uint32_t to, int wv, int t0, int len) const { load(to, wv, t0, len, k, k_row, k_off); }
    __device__ __forceinline__ void load_v(uint32_t to, int wv, int t0, int len) const { load(to, wv, t0, len, v, v_row, v_off); }

private:
    static __device__ __forceinline__ int row_of(int p) { return p / Rows<HD>::CHUNKS; }
    static __device__ __forceinline__ int chunk_of(int p) { return ((p % Rows<HD>::CHUNKS) ^ Rows<HD>::number(row_of(p))) * 16; }
    __device__ __forceinline__ void load(uint32_t to, int wv, int t0, int len, const char *from, int64_t bytes, uint32_t off) const {
        int p = (int)threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = to + (i * WAVES + wv) * Rows<HD>::GROUP;
            const int t = t0 + i * STEP;
            if (t0 + 64 <= len) {
                load_to_lds(from + t * bytes, off, at);
            } else {
                asm volatile("" : "+v"(p));   // formed here: rows and chunks kept for the last keys would cost registers
                load_to_lds(t + row_of(p) < len ? from + t * bytes + off : reinterpret_cast<const char *>(kZeroRow) + chunk_of(p), at);
            }
        }
    }
};

// ---- random numbers ------------------------------------------------------------------------
//
// Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): the
// fewest with which it passes their batteries of tests.
__device__ __forceinline__ u32x4_t philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 7; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return (u32x4_t){c0, c1, c2, c3};
}

struct Random {
    uint32_t k0, k1, offset;
    __device__ __forceinline__ void init(const int64_t *rng) {
        const uint64_t seed = (uint64_t)rng[0];
        k0 = __builtin_amdgcn_readfirstlane((uint32_t)seed);
        k1 = __builtin_amdgcn_readfirstlane((uint32_t)(seed >> 32));
        offset = __builtin_amdgcn_readfirstlane((uint32_t)rng[1]);
    }
    // The bytes of the 16 tokens 32 `block` + 8 w + 4 g + e: byte e of word w.
    __device__ __forceinline__ u32x4_t weights(int block, int g, uint32_t row, uint32_t head) const {
        return philox(2 * block + g, row, head, offset, k0, k1);
    }
};

// The same decisions with tokens in the lanes.  Lane (g, j) gives the words of row j, whose byte e of word w is that of token 8 w +
// 4 g + e; it gets bit r: whether row r keeps token 8 (j % 4) + j & 4 + j / 8 (turned_token).  The bytes are compared four at a time;
// the bits of a row and its tokens are turned by exchanges with the lanes 16, 8, 4, 2 and 1 away.
__device__ __forceinline__ int turned_token(int j) { return 8 * (j & 3) + (j & 4) + (j >> 3); }
template <bool KEEP>   // what depends on the lane alone, in 9 registers
struct Turn {
    int lane;
    static __device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t a, uint32_t b) { return (mask & a) | (~mask & b); }
    template <int CTRL>
    static __device__ __forceinline__ uint32_t from(uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, true); }
    __device__ __forceinline__ uint32_t rows(const u32x4_t &w, uint32_t edge) const {
        int lane = this->lane;
        if constexpr (!KEEP) asm volatile("" : "+v"(lane));
        const uint32_t bytes16 = lane & 16 ? 0x07060302u : 0x05040100u;   // of the pair (lane with bit 4 set : clear)
        const uint32_t bytes8 = lane & 8 ? 0x07030501u : 0x02060004u;     // of the pair (own : other)
        const uint32_t by4 = lane & 4 ? 4 : 28, by2 = lane & 2 ? 2 : 30, by1 = lane & 1 ? 1 : 31, half = lane & 32 ? 0 : 4;
        const uint32_t own4 = lane & 4 ? 0xF0F0F0F0u : 0x0F0F0F0Fu, own2 = lane & 2 ? 0xCCCCCCCCu : 0x33333333u, own1 = lane & 1 ? 0xAAAAAAAAu : 0x55555555u;
        // Bit 7 of each byte: whether it is at least `edge`.  The low 7 bits decide, unless the top ones differ.
        const uint32_t low = (edge & 127) * 0x01010101u, top = edge & 128 ? 0u : 0xFFFFFFFFu;
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = (w[i] | 0x80808080u) - low;
            f[i] = pick(w[i] ^ d, top, d);
        }
        uint32_t x = pick(0x80808080u, f[3], f[2] >> 1);
        x = pick(0xC0C0C0C0u, x, f[1] >> 2);
        x = (pick(0xE0E0E0E0u, x, f[0] >> 3) & 0xF0F0F0F0u) >> half;   // token 8 w + 4 g + e at bit 8 e + 4 g + w
        const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = h[0] | h[1];
        const auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = __builtin_amdgcn_perm(q[1], q[0], bytes16);
        x = __builtin_amdgcn_perm(x, from<0x128>(x), bytes8);                       // 8 lanes round in 16
        uint32_t y = from<0x1B>(from<0x141>(x));                                    // 7 - j in 8, 3 - j in 4: 4 away
        x = pick(own4, x, __builtin_amdgcn_alignbit(y, y, by4));
        y = from<0x4E>(x);                                                          // 2 away
        x = pick(own2, x, __builtin_amdgcn_alignbit(y, y, by2));
        y = from<0xB1>(x);                                                          // 1 away
        return pick(own1, x, __builtin_amdgcn_alignbit(y, y, by1));
    }
};

// ---- places --------------------------------------------------------------------------------

__device__ __forceinline__ int user_len(const TrainArgs &a, int u) { return a.lens ? min(max(a.lens[u], 0), a.L_kv) : a.L_kv; }

struct Place {
    int cand, head, query;
};
// Row r of a user's rows of shared head hk; perm: the user's candidates.
template <class P>
__device__ __forceinline__ Place place_of(const TrainArgs &a, P perm, int hk, int r) {
    const uint32_t per = (uint32_t)(a.G * a.L_q), slot = (uint32_t)r / per, rest = (uint32_t)r - slot * per, gr = rest / (uint32_t)a.L_q;
    return Place{perm[(int)slot], hk * a.G + (int)gr, (int)(rest - gr * (uint32_t)a.L_q)};
}
// Tokens that a query sees.
__device__ __forceinline__ int limit_of(const TrainArgs &a, const Place &p, int len) {
    if (!a.positions) return len;
    const int pos = a.positions[(int64_t)p.cand * a.L_q + p.query];
    return pos < 0 ? 0 : pos < len ? pos + 1 : len;
}

// ---- small calls ---------------------------------------------------------------------------
//
// For few candidates and users every block finds its own place: how many candidates each user has, which tile (or whose
// notes) the block's is, and that user's candidates, in their order.  That takes about as long as reading a table of them,
// and saves the launch that writes it (5 us).

struct LocalLds {
    int count[kLocalUsers], part[kLocalCands / 64], list[kLocalCands];
};

// Counts, by all THREADS threads, whose candidates' users are left in m; then lane u of every wave knows user u's: the
// candidates, tiles and notes before (12, 8 and 12 bits) and rows.
template <int THREADS>
struct Local {
    int m[kLocalCands / THREADS], before, rows, len;
    __device__ __forceinline__ void count(const TrainArgs &a, LocalLds &s) {
        const int tid = (int)threadIdx.x, lane = tid & 63;
        uint32_t err = 0;
#pragma unroll
        for (int i = 0; i < kLocalCands / THREADS; ++i) m[i] = tid + i * THREADS < a.B_c ? a.map[tid + i * THREADS] : -1;
        len = lane < a.B_u ? user_len(a, lane) : 0;
        if (lane < a.B_u && a.lens && a.lens[lane] != len) err = kTrainStLens;
        if (tid < kLocalUsers) s.count[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLocalCands / THREADS; ++i) {
            if (m[i] >= 0 && m[i] < a.B_u) atomicAdd(&s.count[m[i]], 1);
            else if (m[i] != -1) err |= kTrainStMap;
        }
        if (err) atomicOr(a.status, err);
        __syncthreads();
        const int n = lane < a.B_u ? s.count[lane] : 0;
        rows = n * a.G * a.L_q;
        const int own = n | (rows + kTileRows - 1) / kTileRows << 12 | ((rows + 63) / 64) << 20;
        before = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(before, d);
            if (lane >= d) before += x;
        }
        before -= own;
    }
    // The user whose tile this is; user -1 if there is none.
    __device__ __forceinline__ TileEntry tile(int at) const {
        const int first = before >> 12 & 255, n = (rows + kTileRows - 1) / kTileRows;
        const uint64_t here = __ballot(at >= first && at < first + n);
        if (!here) return TileEntry{-1, 0, 0, 0, 0, 0, {0, 0}};
        const int u = __ffsll((unsigned long long)here) - 1, b = __builtin_amdgcn_readlane(before, u), row = (at - (b >> 12 & 255)) * kTileRows;
        return TileEntry{u, row, b & 4095, __builtin_amdgcn_readlane(rows, u), __builtin_amdgcn_readlane(len, u), (b >> 20) + row / 64, {0, 0}};
    }
    // All rows of user u.
    __device__ __forceinline__ ChunkEntry chunk(int u) const {
        return ChunkEntry{u, __builtin_amdgcn_readlane(before, u) >> 20, (__builtin_amdgcn_readlane(rows, u) + 63) / 64, -1, __builtin_amdgcn_readlane(len, u), {0, 0, 0}};
    }
    // User u's candidates to s.list.
    __device__ __forceinline__ void list(const TrainArgs &a, LocalLds &s, int u) const {
        const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
        uint64_t mine[kLocalCands / THREADS];
#pragma unroll
        for (int i = 0; i < kLocalCands / THREADS; ++i) {
            mine[i] = __ballot(m[i] == u);
            if (lane == 0) s.part[i * (THREADS / 64) + wv] = __popcll(mine[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLocalCands / THREADS; ++i) {
            int at = __popcll(mine[i] & ((1ull << lane) - 1));
            for (int w = 0; w < i * (THREADS / 64) + wv; ++w) at += s.part[w];
            if (m[i] == u) s.list[at] = tid + i * THREADS;
        }
        __syncthreads();
    }
};

// O = 0 and lse = -inf, or dQ = 0, of candidates whose map entry is no user: block `block` of a.pads.  A wave looks at 64
// candidates; where there are more waves than that, several share those of 64.
__device__ __forceinline__ void fill_padding(const TrainArgs &a, int head_dim, bool backward, int block) {
    const int n = a.H_q * a.L_q, waves = a.pads * (int)blockDim.x / 64, groups = max(1, (a.B_c + 63) / 64), share = max(1, waves / groups);
    const int wave = block * (int)blockDim.x / 64 + ((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63, first = wave % share * 64 + lane, step = 64 * share;
    if (wave >= waves / share * share) return;
    for (int b0 = wave / share * 64; b0 < a.B_c; b0 += waves / share * 64) {
        const int u = b0 + lane < a.B_c ? a.map[b0 + lane] : 0;
        uint64_t none = __ballot(u < 0 || u >= a.B_u);
        while (none) {
            const int b = b0 + __ffsll((unsigned long long)none) - 1;
            none &= none - 1;
            uint16_t *to = backward ? a.dQ + b * a.dq_cand : a.O + b * a.o_cand;
            const int64_t head = backward ? a.dq_head : a.o_head, query = backward ? a.dq_query : a.o_query;
            const int shift = head_dim == 128 ? 4 : 3;
            for (int64_t i = first; i < (int64_t)n << shift; i += step) {
                const int r = (int)(i >> shift), h = r / a.L_q;
                *reinterpret_cast<u32x4_t *>(to + h * head + (r - h * a.L_q) * query + 8 * ((int)i & ((1 << shift) - 1))) = (u32x4_t){0, 0, 0, 0};
            }
            if (!backward)
                for (int i = first; i < n; i += step) a.lse[(int64_t)b * n + i] = neg_inf();
        }
    }
}

// Blocks go round the 8 dies in turn; runs of 8 (or 4) neighbouring units, which share what they read, go to one
// die: 70:1 forward 155 -> 151 us, 10:1 dK and dV 77 -> 65 (dQ 46 -> 50).  Few units are dealt one by one, so that all dies
// have some.  Whole eighths of the units to each die leave the dies uneven where units differ (70:1 dK and dV 462).  Unit
// of this block among n, or -1.
__device__ __forceinline__ int unit_of(int block, int n) {
    const int log_run = n >= 512 ? 3 : n >= 128 ? 2 : 0, i = block >> 3;
    const int at = ((((i >> log_run) << 3) + (block & 7)) << log_run) + (i & ((1 << log_run) - 1));
    return at < n ? at : -1;
}
// Blocks for n units.
inline unsigned blocks_of(int64_t n) { return (unsigned)((n + 63) / 64 * 64); }
// Units of tiles of rows: eight tiles (or the last ones) of a shared head, the same of the next head, and so on; then the
// next eight, since the grouping puts the tiles in the order of their work; then the next part of the keys.
struct TileUnit {
    int tile, hk, split;
};
__device__ __forceinline__ TileUnit tile_unit(const TrainArgs &a, int unit) {
    const int all = a.tiles * a.H_kv, x = unit % all, first = x / (8 * a.H_kv) * 8, n = min(8, a.tiles - first), y = x - first * a.H_kv;
    return TileUnit{first + y % n, y / n, unit / all};
}

// Element quads 2 p and 2 p + 1 of a result column, rounded: 8 consecutive rows 16 p + 8 g .. of it for this lane.
__device__ __forceinline__ u32x4_t eight_rows(const f32x16_t &x, int p, float by) {
    const uint32_t a0 = pack_bf16x2(x[8 * p] * by, x[8 * p + 1] * by), a1 = pack_bf16x2(x[8 * p + 2] * by, x[8 * p + 3] * by);
    const uint32_t b0 = pack_bf16x2(x[8 * p + 4] * by, x[8 * p + 5] * by), b1 = pack_bf16x2(x[8 * p + 6] * by, x[8 * p + 7] * by);
    const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false), s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
    return (u32x4_t){s0[0], s1[0], s0[1], s1[1]};
}

}  // namespace ikbo
