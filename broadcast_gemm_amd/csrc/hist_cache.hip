// hist_cache.hip -- writing rows of keys and values into the 4-bit cache, and reading them back
// (ikbo_kv4_write, ikbo_kv4_read).  The tile of a (page, head) is described in ikbo.h.
//
// Write: a block takes 64 token rows of one head (16 where 64 would leave most of the chip idle).
// 8 elements of a row (one thread, 16 or 32 bytes) become 4 bytes of codes; 4 neighbouring threads hold the
// 32 elements of one scale and share their largest magnitude by two lane exchanges.  The scale is a power
// of two, so the hardware's conversion (x / 2^e to the nearest code, ties to even, never beyond 6) is
// exact: the stored bytes are a function of the inputs alone.  K codes are rows of the tile and are
// stored as they come.  V codes stand token by token behind each element pair, so they go through LDS, and
// each thread stores the tokens of one element pair: 16 or 4 bytes at once where neighbouring rows have
// neighbouring slots in a page, single bytes otherwise.
//
// Read: for K a thread takes 8 elements of a row, for V an element pair of 4 rows: one access where their
// slots are neighbours, and the lanes of a wave, neighbouring pairs, write whole rows.
//
// Both are bound by their bytes once there are enough rows, and by a launch and two dependent reads where there are
// few.  16381 tokens of 8 heads of 128, bf16: write 20 us (67 MB in, 18 out: 4.3 TB/s), read 22 us (3.9 TB/s);
// 59 tokens of 4 heads: 3.5 and 3.8 us.
#include "hist_internal.h"

#include "lce_device.h"

namespace ikbo {
namespace {

constexpr int kThreads = 256;
__device__ __forceinline__ int scale_place(int t) { return (t & 48) + 4 * (t & 3) + ((t >> 2) & 3); }

// 8 elements of a row as they stand in memory.
template <bool F32> struct Eight;
template <> struct Eight<false> {
    u32x4_t w;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        w = *reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(base) + at);
    }
    __device__ __forceinline__ void clear() { w = (u32x4_t){0, 0, 0, 0}; }
    // The largest magnitude, as the bits of a float32.
    __device__ __forceinline__ uint32_t top() const {
        typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
        u16x2_t m = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[e] & 0x7FFF7FFFu));
        return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
    }
    // What the cache cannot hold: NaN becomes 0 and infinity the largest finite value.
    __device__ __forceinline__ void mend() {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t y = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t v = (w[e] >> (16 * k)) & 0xFFFFu, m = v & 0x7FFFu;
                y |= (m > 0x7F80u ? 0u : m == 0x7F80u ? v - 1u : v) << (16 * k);
            }
            w[e] = y;
        }
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (uint32_t)w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (uint32_t)w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (uint32_t)w[2]), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (uint32_t)w[3]), scale, 3);
    }
};
template <> struct Eight<true> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        const u32x4_t *p = reinterpret_cast<const u32x4_t *>(static_cast<const float *>(base) + at);
        const u32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { w[e] = a[e]; w[4 + e] = b[e]; }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 0;
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, w[e] & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ void mend() {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = w[e] & 0x7FFFFFFFu;
            w[e] = m > 0x7F800000u ? 0u : m == 0x7F800000u ? w[e] - 1u : w[e];
        }
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        auto x = [&](int e) { return __builtin_bit_cast(float, w[e]); };
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x(0), x(1), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x(2), x(3), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x(4), x(5), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x(6), x(7), scale, 3);
    }
};

// 8 elements of one row as 4 bytes of codes; *scale is the byte of their 32 elements (the threads
// 4q .. 4q+3 hold them).
template <bool F32>
__device__ __forceinline__ uint32_t encode8(Eight<F32> &x, uint32_t *scale, bool *odd) {
    if (x.top() >= 0x7F800000u) {
        *odd = true;
        x.mend();
    }
    uint32_t top = x.top();
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));   // lane ^ 1
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));   // lane ^ 2
    int e2 = (int)(top >> 23) - 127 - 2 + ((top & 0x7FFFFFu) > 0x400000u);   // top <= 6 * 2^e2
    e2 = e2 < -125 ? -125 : e2 > 125 ? 125 : e2;
    *scale = (uint32_t)(e2 + 127);
    return x.codes(__builtin_bit_cast(float, *scale << 23));
}

template <int HD, bool F32, int kRows>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(ikbo_kv4_rows_args a) {
    constexpr int CH = HD / 8;           // threads per row
    constexpr int PAIRS = HD / 2;
    constexpr int TILE = 68 * HD;
    constexpr int VROW = kRows + 4;      // bytes per element pair in LDS
    __shared__ int s_slot[kRows];
    __shared__ uint32_t s_v[PAIRS * VROW / 4];
    __shared__ uint32_t s_flag;
    __shared__ uint64_t s_next;
    const int tid = (int)threadIdx.x, h = (int)blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * kRows;
    const int nr = (int)min((int64_t)kRows, a.T - r0);
    // All of the thread's rows are on their way before their slots are known.
    constexpr int ITEMS = kRows * CH, TURNS = (ITEMS + kThreads - 1) / kThreads;
    Eight<F32> kx[TURNS], vx[TURNS];
#pragma unroll
    for (int y = 0; y < TURNS; ++y) {
        const int x = tid + y * kThreads, r = x / CH, c = x % CH;
        kx[y].clear();
        vx[y].clear();
        if (x < ITEMS && r < nr) {
            kx[y].load(a.k, (r0 + r) * a.k_token + h * a.k_head + 8 * c);
            vx[y].load(a.v, (r0 + r) * a.v_token + h * a.v_head + 8 * c);
        }
    }
    if (tid == 0) s_flag = 0;
    __syncthreads();
    if (tid < 64) {
        int slot = tid < nr ? a.slots[r0 + tid] : -1;
        if (slot < -1 || slot >= a.num_pages * IKBO_KV4_PAGE) {
            if (h == 0) atomicOr(&s_flag, kStPage);
            slot = -1;
        }
        if (tid < kRows) s_slot[tid] = slot;
        // Bit r: row r stands right behind row r - 1 in the same page.
        const int before = __shfl_up(slot, 1);
        const uint64_t next = __ballot(tid > 0 && before >= 0 && slot == before + 1 && slot % IKBO_KV4_PAGE != 0);
        if (tid == 0) s_next = next;
    }
    __syncthreads();
    char *tiles = static_cast<char *>(a.tiles);
    uint8_t *vb = reinterpret_cast<uint8_t *>(s_v);
#pragma unroll
    for (int y = 0; y < TURNS; ++y) {
        const int x = tid + y * kThreads, r = x / CH, c = x % CH;
        if (x >= ITEMS) break;
        const int slot = s_slot[r];
        const bool live = slot >= 0;
        uint32_t ks, vs;
        bool odd = false;
        const uint32_t kw = encode8(kx[y], &ks, &odd), vw = encode8(vx[y], &vs, &odd);
        if (odd && live) atomicOr(&s_flag, kStNonfinite);
        if (live) {
            char *tile = tiles + ((int64_t)(slot / IKBO_KV4_PAGE) * a.H_kv + h) * TILE;
            const int t = slot % IKBO_KV4_PAGE;
            *reinterpret_cast<uint32_t *>(tile + t * PAIRS + 4 * c) = kw;
            if (c % 4 == 0) {
                tile[64 * HD + (c / 4) * 64 + scale_place(t)] = (char)ks;
                tile[66 * HD + (c / 4) * 64 + t] = (char)vs;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) vb[(4 * c + e) * VROW + r] = (uint8_t)(vw >> (8 * e));
        }
    }
    __syncthreads();
    // The V codes of one element pair, this thread's share of the rows (at most 16): the stores may have any
    // alignment, and a run within a page stays within the pair's 64 bytes.
    constexpr int PART = kRows * PAIRS / kThreads;
    const int pair = tid % PAIRS, first = tid / PAIRS * PART;
    const uint64_t next = s_next;
    auto together = [&](int r, int n) { return ((next >> r) & ((1ull << n) - 2)) == (1ull << n) - 2; };   // rows r .. r + n - 1
    auto place = [&](int slot) {
        return tiles + ((int64_t)(slot / IKBO_KV4_PAGE) * a.H_kv + h) * TILE + PAIRS * 64 + pair * 64 + slot % IKBO_KV4_PAGE;
    };
    const uint8_t *from = vb + pair * VROW + first;
    if (PART == 16 && together(first, 16)) {
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const uint32_t *>(from)[e];
        __builtin_memcpy(place(s_slot[first]), &w, 16);
    } else {
        constexpr int STEP = PART < 4 ? PART : 4;
#pragma unroll
        for (int r = 0; r < PART; r += STEP) {
            if (STEP == 4 && together(first + r, 4)) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(from + r);
                __builtin_memcpy(place(s_slot[first + r]), &w, 4);
            } else {
#pragma unroll
                for (int e = 0; e < STEP; ++e) {
                    const int slot = s_slot[first + r + e];
                    if (slot >= 0) *place(slot) = (char)from[r + e];
                }
            }
        }
    }
    if (tid == 0 && s_flag) atomicOr(a.status, s_flag);
}

template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, const uint32_t (&w)[4]) {
    if constexpr (F32) {
        u32x4_t *p = reinterpret_cast<u32x4_t *>(static_cast<float *>(base) + at);
        p[0] = (u32x4_t){w[0] << 16, w[0] & 0xFFFF0000u, w[1] << 16, w[1] & 0xFFFF0000u};
        p[1] = (u32x4_t){w[2] << 16, w[2] & 0xFFFF0000u, w[3] << 16, w[3] & 0xFFFF0000u};
    } else {
        *reinterpret_cast<u32x4_t *>(static_cast<uint16_t *>(base) + at) = (u32x4_t){w[0], w[1], w[2], w[3]};
    }
}

template <bool F32>
__device__ __forceinline__ void store2(void *base, int64_t at, uint32_t w) {
    if constexpr (F32) *reinterpret_cast<u32x2_t *>(static_cast<float *>(base) + at) = (u32x2_t){w << 16, w & 0xFFFF0000u};
    else *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + at) = w;
}

template <int HD, bool F32>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(ikbo_kv4_rows_args a) {
    constexpr int CH = HD / 8, PAIRS = HD / 2, TILE = 68 * HD;
    const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int h = (int)blockIdx.y, n_slots = a.num_pages * IKBO_KV4_PAGE;
    auto tile_of = [&](int slot) {
        return static_cast<const char *>(a.tiles) + ((int64_t)(slot / IKBO_KV4_PAGE) * a.H_kv + h) * TILE;
    };
    const int64_t r = x / CH;
    if (r < a.T) {
        const int c = (int)(x % CH), slot = a.slots[r];
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1 && c == 0 && h == 0) atomicOr(a.status, kStPage);
        } else if (a.k) {
            const char *tile = tile_of(slot);
            const int t = slot % IKBO_KV4_PAGE;
            const uint32_t codes = *reinterpret_cast<const uint32_t *>(tile + t * PAIRS + 4 * c);
            const float s = __builtin_bit_cast(float, (uint32_t)(uint8_t)tile[64 * HD + (c / 4) * 64 + scale_place(t)] << 23);
            uint32_t w[4];
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
            store8<F32>(a.k, r * a.k_token + h * a.k_head + 8 * c, w);
        }
    }
    const int64_t r4 = x / PAIRS * 4;
    if (!a.v || r4 >= a.T) return;
    const int pair = (int)(x % PAIRS);
    int slot[4];
    bool near = true;   // four neighbouring slots of one page
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        slot[e] = r4 + e < a.T ? a.slots[r4 + e] : -1;
        if (slot[e] >= n_slots) slot[e] = -1;
        near = near && slot[0] >= 0 && slot[e] == slot[0] + e && slot[0] % IKBO_KV4_PAGE <= IKBO_KV4_PAGE - 4;
    }
    const int64_t v_at = 32 * HD + pair * 64, s_at = 66 * HD + (pair / 16) * 64;
    uint32_t codes = 0, scales = 0;
    if (near) {
        const char *tile = tile_of(slot[0]) + slot[0] % IKBO_KV4_PAGE;
        __builtin_memcpy(&codes, tile + v_at, 4);     // any alignment
        __builtin_memcpy(&scales, tile + s_at, 4);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (slot[e] >= 0) {
                const char *tile = tile_of(slot[e]) + slot[e] % IKBO_KV4_PAGE;
                codes |= (uint32_t)(uint8_t)tile[v_at] << (8 * e);
                scales |= (uint32_t)(uint8_t)tile[s_at] << (8 * e);
            }
    }
    auto put = [&](int e, auto w) {
        if (slot[e] >= 0) store2<F32>(a.v, (r4 + e) * a.v_token + h * a.v_head + 2 * pair, __builtin_bit_cast(uint32_t, w));
    };
    put(0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __builtin_bit_cast(float, (scales & 0xFFu) << 23), 0));
    put(1, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __builtin_bit_cast(float, (scales >> 8 & 0xFFu) << 23), 1));
    put(2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __builtin_bit_cast(float, (scales >> 16 & 0xFFu) << 23), 2));
    put(3, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __builtin_bit_cast(float, (scales >> 24) << 23), 3));
}

template <int HD, bool F32>
hipError_t launch_write(const ikbo_kv4_rows_args &a, hipStream_t s) {
    // 64 rows make the wide stores of V; below two blocks for each of 256 CUs the time of one block counts, and 16
    // rows take less of it.  In us with 64 and 16 rows: 59 tokens of 4 heads 5.8 and 3.5, 16381 of 8 heads 20.4 and 23.3.
    const int64_t wide = (int64_t)((a.T + 63) / 64) * a.H_kv;
    if (wide >= 512) hipLaunchKernelGGL((kv4_write_kernel<HD, F32, 64>), dim3((unsigned)((a.T + 63) / 64), (unsigned)a.H_kv), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kv4_write_kernel<HD, F32, 16>), dim3((unsigned)((a.T + 15) / 16), (unsigned)a.H_kv), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <int HD, bool F32>
hipError_t launch_read(const ikbo_kv4_rows_args &a, hipStream_t s) {
    const int64_t threads = ((int64_t)a.T + 3) / 4 * (HD / 2);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)a.H_kv);
    hipLaunchKernelGGL((kv4_read_kernel<HD, F32>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

// A launch counts its threads in 32 bits (more are dropped without an error): 2^27 rows at a time are 2^31 of the read.
template <class Launch>
hipError_t by_parts(const ikbo_kv4_rows_args &a, hipStream_t s, Launch launch) {
    constexpr int64_t kMost = 1ll << 27;
    const int size = a.dtype == IKBO_DTYPE_F32 ? 4 : 2;
    for (int64_t r = 0; r < a.T; r += kMost) {
        ikbo_kv4_rows_args part = a;
        part.T = (int)(a.T - r < kMost ? a.T - r : kMost);
        part.slots += r;
        part.k = beyond(a.k, r * a.k_token, size);
        part.v = beyond(a.v, r * a.v_token, size);
        const hipError_t e = launch(part, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_kv4_write(const ikbo_kv4_rows_args &a, hipStream_t s) {
    const bool f = a.dtype == IKBO_DTYPE_F32;
    if (a.head_dim == 128) return by_parts(a, s, f ? launch_write<128, true> : launch_write<128, false>);
    return by_parts(a, s, f ? launch_write<64, true> : launch_write<64, false>);
}

hipError_t launch_kv4_read(const ikbo_kv4_rows_args &a, hipStream_t s) {
    const bool f = a.dtype == IKBO_DTYPE_F32;
    if (a.head_dim == 128) return by_parts(a, s, f ? launch_read<128, true> : launch_read<128, false>);
    return by_parts(a, s, f ? launch_read<64, true> : launch_read<64, false>);
}

}  // namespace ikbo
