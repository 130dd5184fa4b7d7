// dropout.hip -- dropout of activations from the counter-based generator (ikbo_dropout): y = residual + x / (1 - p)
// where an element stays.  Nothing is stored: the gradient is the same call on the gradient.
//
// A thread takes 8 elements, which one generator call decides with 16 bits each.  Each element is read and written
// once; that bounds it: 15.7 million bf16 with residual (94 MB, most of it in the caches) 15.4 us, 63 million float32
// (503 MB) 89 us, 5.6 TB/s, where a copy of 4 GiB reaches 4.8.
#include "train_device.h"

namespace ikbo {
namespace {

template <bool F32>
struct Eight {   // 8 elements, in 16-byte pieces
    u32x4_t v[F32 ? 2 : 1];
    __device__ __forceinline__ float at(int i) const {
        if constexpr (F32) return __builtin_bit_cast(float, (uint32_t)v[i >> 2][i & 3]);
        const uint32_t w = v[0][i >> 1];
        return __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

template <bool F32>
__device__ __forceinline__ float one(const void *p, int64_t i) {
    if constexpr (F32) return static_cast<const float *>(p)[i];
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(256) dropout_kernel(const void *x, const void *residual, void *y, const int64_t *rng, int64_t n, uint32_t edge, float keep) {
    constexpr int SIZE = F32 ? 4 : 2;
    Random rnd;
    rnd.init(rng);
    for (int64_t c = (int64_t)blockIdx.x * 256 + (int)threadIdx.x; c * 8 < n; c += (int64_t)gridDim.x * 256) {
        const bool whole = WIDE && c * 8 + 8 <= n;
        float v[8], r[8];
        const int64_t left = n - c * 8;
        if (whole) {
            const Eight<F32> in = *reinterpret_cast<const Eight<F32> *>(static_cast<const char *>(x) + c * 8 * SIZE);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = in.at(i);
            if (residual) {
                const Eight<F32> add = *reinterpret_cast<const Eight<F32> *>(static_cast<const char *>(residual) + c * 8 * SIZE);
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = add.at(i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = i < left ? one<F32>(x, c * 8 + i) : 0.f;
                r[i] = residual && i < left ? one<F32>(residual, c * 8 + i) : 0.f;
            }
        }
        const u32x4_t w = philox((uint32_t)c, (uint32_t)((uint64_t)c >> 32), 0xFFFFFFFFu, rnd.offset, rnd.k0, rnd.k1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float kept = ((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu) >= edge ? v[i] * keep : 0.f;
            v[i] = residual ? r[i] + kept : kept;
        }
        if (whole) {
            Eight<F32> out;
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) out.v[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) out.v[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            }
            *reinterpret_cast<Eight<F32> *>(static_cast<char *>(y) + c * 8 * SIZE) = out;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= left) break;
                if constexpr (F32) static_cast<float *>(y)[c * 8 + i] = v[i];
                else static_cast<uint16_t *>(y)[c * 8 + i] = (uint16_t)(pack_bf16x2(v[i], 0.f) & 0xFFFFu);
            }
        }
    }
}

template <bool F32>
hipError_t launch(const ikbo_dropout_args &a, uint32_t edge, float keep, hipStream_t s) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.y);
    const int64_t calls = (a.n + 7) / 8, blocks = (calls + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20));
    if (any & 15) hipLaunchKernelGGL((dropout_kernel<F32, false>), grid, dim3(256), 0, s, a.x, a.residual, a.y, a.rng, a.n, edge, keep);
    else hipLaunchKernelGGL((dropout_kernel<F32, true>), grid, dim3(256), 0, s, a.x, a.residual, a.y, a.rng, a.n, edge, keep);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const ikbo_dropout_args &a, uint32_t edge, hipStream_t s) {
    const float keep = (float)(65536.0 / (65536 - (int)edge));
    return a.dtype == IKBO_DTYPE_F32 ? launch<true>(a, edge, keep, s) : launch<false>(a, edge, keep, s);
}

}  // namespace ikbo
