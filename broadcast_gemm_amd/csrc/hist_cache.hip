// hist_cache.hip -- writing rows of keys and values into the 4-bit cache, and reading them back
// (ikbo_kv4_write, ikbo_kv4_read).  The tile of a (page, head) is described in ikbo.h.
//
// Write: a block takes 64 token rows of one head (16 where 64 would leave most of the chip idle).  8 elements of a row (one thread, 16 or 32 bytes)
// become 4 bytes of codes; 4 neighbouring threads hold the 32 elements of one scale and share their
// largest magnitude by two lane exchanges.  The scale is a power of two, so x / 2^e and the hardware's
// conversion to the nearest code (ties to even) are exact: the stored bytes are a function of the inputs
// alone.  K codes are rows of the tile and are stored as they come.  V codes stand token by token
// behind each element pair, so they go through LDS, and each thread stores the tokens of one element
// pair: 16 or 4 bytes at once where neighbouring rows have neighbouring slots in a tile, single bytes
// otherwise.
#include "hist_internal.h"

#include "lce_device.h"

namespace ikbo {
namespace {

constexpr int kThreads = 256;
__device__ __forceinline__ int scale_place(int t) { return (t & 48) + 4 * (t & 3) + ((t >> 2) & 3); }

template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&x)[8]) {
    if constexpr (F32) {
        const u32x4_t *p = reinterpret_cast<const u32x4_t *>(static_cast<const float *>(base) + at);
        const u32x4_t a = p[0], b = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = __builtin_bit_cast(float, (uint32_t)a[e]);
            x[4 + e] = __builtin_bit_cast(float, (uint32_t)b[e]);
        }
    } else {
        const u32x4_t a = *reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(base) + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __builtin_bit_cast(float, a[e] << 16);
            x[2 * e + 1] = __builtin_bit_cast(float, a[e] & 0xFFFF0000u);
        }
    }
}

// 8 elements of one row as 4 bytes of codes; *scale is the byte of their 32 elements (the threads
// 4q .. 4q+3 hold them).
__device__ __forceinline__ uint32_t encode8(float (&x)[8], uint32_t *scale, bool *odd) {
    constexpr float kMost = 3.3895313892515355e38f;   // beyond the largest value the cache holds
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (x[e] != x[e]) { x[e] = 0.f; *odd = true; }
        if (__builtin_fabsf(x[e]) > kMost) {
            *odd = *odd || __builtin_isinf(x[e]);
            x[e] = __builtin_copysignf(kMost, x[e]);
        }
        top = fmaxf(top, __builtin_fabsf(x[e]));
    }
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    const uint32_t bits = __builtin_bit_cast(uint32_t, top);
    int e2 = (int)(bits >> 23) - 127 - 2 + ((bits & 0x7FFFFFu) > 0x400000u);   // top <= 6 * 2^e2
    e2 = e2 < -125 ? -125 : e2 > 125 ? 125 : e2;
    *scale = (uint32_t)(e2 + 127);
    const float inv = __builtin_bit_cast(float, (uint32_t)(127 - e2) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * inv, x[1] * inv, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * inv, x[3] * inv, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * inv, x[5] * inv, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * inv, x[7] * inv, 1.0f, 3);
    return w;
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
    const int tid = (int)threadIdx.x, h = (int)blockIdx.y;
    const int64_t r0 = (int64_t)blockIdx.x * kRows;
    const int nr = (int)min((int64_t)kRows, a.T - r0);
    if (tid == 0) s_flag = 0;
    __syncthreads();
    if (tid < kRows) {
        int slot = tid < nr ? a.slots[r0 + tid] : -1;
        if (slot < -1 || slot >= a.num_pages * IKBO_KV4_PAGE) {
            if (h == 0) atomicOr(&s_flag, kStPage);
            slot = -1;
        }
        s_slot[tid] = slot;
    }
    __syncthreads();
    char *tiles = static_cast<char *>(a.tiles);
    uint8_t *vb = reinterpret_cast<uint8_t *>(s_v);
    for (int x = tid; x < kRows * CH; x += kThreads) {
        const int r = x / CH, c = x % CH;
        const int slot = s_slot[r];
        const bool live = slot >= 0;
        float kx[8] = {}, vx[8] = {};
        if (live) {
            load8<F32>(a.k, (r0 + r) * a.k_token + h * a.k_head + 8 * c, kx);
            load8<F32>(a.v, (r0 + r) * a.v_token + h * a.v_head + 8 * c, vx);
        }
        uint32_t ks, vs;
        bool odd = false;
        const uint32_t kw = encode8(kx, &ks, &odd), vw = encode8(vx, &vs, &odd);
        if (odd) atomicOr(&s_flag, kStNonfinite);
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
    // The V codes of one element pair, this thread's share of the rows.
    constexpr int PART = kRows * PAIRS / kThreads;   // rows per thread: at most 16
    const int pair = tid % PAIRS, first = tid / PAIRS * PART;
    for (int r = first; r < first + PART;) {
        const int slot = s_slot[r];
        if (slot < 0) { ++r; continue; }
        const int t = slot % IKBO_KV4_PAGE;
        char *to = tiles + ((int64_t)(slot / IKBO_KV4_PAGE) * a.H_kv + h) * TILE + PAIRS * 64 + pair * 64 + t;
        int run = 1;
        while (run < 16 && r + run < first + PART && s_slot[r + run] == slot + run && (t + run) % 16 != 0) ++run;
        const uint8_t *from = vb + pair * VROW + r;
        if (run == 16) {   // then t % 16 == 0
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const uint32_t *>(from)[e];
            *reinterpret_cast<u32x4_t *>(to) = w;
        } else {
            for (int e = 0; e < run;) {
                if ((t + e) % 4 == 0 && e + 4 <= run) {
                    const uint32_t w = from[e] | (from[e + 1] << 8) | (from[e + 2] << 16) | ((uint32_t)from[e + 3] << 24);
                    *reinterpret_cast<uint32_t *>(to + e) = w;
                    e += 4;
                } else {
                    to[e] = (char)from[e];
                    ++e;
                }
            }
        }
        r += run;
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

// Read: a thread takes 8 elements of one row of K and of V.
template <int HD, bool F32>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(ikbo_kv4_rows_args a) {
    constexpr int CH = HD / 8, PAIRS = HD / 2, TILE = 68 * HD;
    const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = x / CH;
    const int c = (int)(x % CH), h = (int)blockIdx.y;
    if (r >= a.T) return;
    const int slot = a.slots[r];
    if (slot < 0 || slot >= a.num_pages * IKBO_KV4_PAGE) {
        if (slot != -1 && c == 0 && h == 0) atomicOr(a.status, kStPage);
        return;
    }
    const char *tile = static_cast<const char *>(a.tiles) + ((int64_t)(slot / IKBO_KV4_PAGE) * a.H_kv + h) * TILE;
    const int t = slot % IKBO_KV4_PAGE;
    auto values = [&](uint32_t codes, uint32_t scale, uint32_t (&w)[4]) {
        const float s = __builtin_bit_cast(float, scale << 23);
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
    };
    uint32_t w[4];
    if (a.k) {
        values(*reinterpret_cast<const uint32_t *>(tile + t * PAIRS + 4 * c),
               (uint8_t)tile[64 * HD + (c / 4) * 64 + scale_place(t)], w);
        store8<F32>(a.k, r * a.k_token + h * a.k_head + 8 * c, w);
    }
    if (a.v) {
        uint32_t codes = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) codes |= (uint32_t)(uint8_t)tile[PAIRS * 64 + (4 * c + e) * 64 + t] << (8 * e);
        values(codes, (uint8_t)tile[66 * HD + (c / 4) * 64 + t], w);
        store8<F32>(a.v, r * a.v_token + h * a.v_head + 8 * c, w);
    }
}

template <int HD, bool F32>
hipError_t launch_write(const ikbo_kv4_rows_args &a, hipStream_t s) {
    // 64 rows make the wide stores of V; below two blocks for each of 256 CUs the time of one block counts,
    // and 16 rows take a third of it (59 tokens, 4 heads: 12 against 4 us).
    const int64_t wide = (int64_t)((a.T + 63) / 64) * a.H_kv;
    if (wide >= 512) hipLaunchKernelGGL((kv4_write_kernel<HD, F32, 64>), dim3((unsigned)((a.T + 63) / 64), (unsigned)a.H_kv), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kv4_write_kernel<HD, F32, 16>), dim3((unsigned)((a.T + 15) / 16), (unsigned)a.H_kv), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_write(const ikbo_kv4_rows_args &a, hipStream_t s) {
    const bool f = a.dtype == IKBO_DTYPE_F32;
    if (a.head_dim == 128) return f ? launch_write<128, true>(a, s) : launch_write<128, false>(a, s);
    return f ? launch_write<64, true>(a, s) : launch_write<64, false>(a, s);
}

hipError_t launch_kv4_read(const ikbo_kv4_rows_args &a, hipStream_t s) {
    const int64_t threads = (int64_t)a.T * (a.head_dim / 8);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)a.H_kv);
    auto go = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, s, a); };
    const bool f = a.dtype == IKBO_DTYPE_F32;
    if (a.head_dim == 128) f ? go(kv4_read_kernel<128, true>) : go(kv4_read_kernel<128, false>);
    else f ? go(kv4_read_kernel<64, true>) : go(kv4_read_kernel<64, false>);
    return hipGetLastError();
}

}  // namespace ikbo
