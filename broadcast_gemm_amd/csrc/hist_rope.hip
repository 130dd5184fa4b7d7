// hist_rope.hip -- rotary positions of queries and keys (ikbo_rope).
//
// Pair i of every head of token t turns by the angle p freq[i], p = positions[t].  The angle in
// turns, p freq[i] / 2 pi, is formed in float64 and its nearest whole number taken off before it is
// rounded to float32: at p = 10^6 and freq = 1 a float32 angle would be off by 0.03 radians, this one
// is off by 2^-25 turns.  Sine and cosine depend on the token and the pair only, so a block computes
// them once for its tokens into LDS and all heads of q and k read them from there: the kernel is bound
// by reading and writing q and k once: 16381 tokens of 32 + 8 heads of 128 in bf16 take 62 us (335 MB, 5.4 TB/s), 15
// tokens of 4 + 4 heads 2.7 us (launch, sines, one access).
//
// VEC elements (16 bytes) per thread and access where the heads allow it (rot_dim, head_dim and the
// strides whole multiples of VEC, 16-byte aligned bases); VEC = 1 otherwise.
#include "hist_internal.h"

#include <algorithm>

#include "lce_device.h"

namespace ikbo {
namespace {

constexpr int kThreads = 256;

template <int BYTES> struct Raw;
template <> struct Raw<16> { typedef u32x4_t type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

// VEC elements of type bf16 (F32 = false) or float32.
template <bool F32, int VEC>
struct Vec {
    typedef typename Raw<VEC * (F32 ? 4 : 2)>::type raw_t;
    static constexpr int SIZE = F32 ? 4 : 2;
    float x[VEC];
    __device__ __forceinline__ void load(const char *p) {
        const raw_t r = *reinterpret_cast<const raw_t *>(p);
        if constexpr (F32 && VEC == 1) x[0] = __builtin_bit_cast(float, r);
        else if constexpr (F32) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = __builtin_bit_cast(float, (uint32_t)r[e]);
        } else if constexpr (VEC == 1) x[0] = __builtin_bit_cast(float, (uint32_t)r << 16);
        else {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                x[e] = __builtin_bit_cast(float, r[e / 2] << 16);
                x[e + 1] = __builtin_bit_cast(float, r[e / 2] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void store(char *p) const {
        raw_t r;
        if constexpr (F32 && VEC == 1) r = __builtin_bit_cast(uint32_t, x[0]);
        else if constexpr (F32) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[e] = __builtin_bit_cast(uint32_t, x[e]);
        } else if constexpr (VEC == 1) r = (uint16_t)pack_bf16x2(x[0], 0.f);
        else {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) r[e / 2] = pack_bf16x2(x[e], x[e + 1]);
        }
        *reinterpret_cast<raw_t *>(p) = r;
    }
};

// Spelt out so that every variant rounds alike.
__device__ __forceinline__ void turn(float a, float b, const float2 &t, float &x, float &y) {
    x = __builtin_fmaf(a, t.x, -(b * t.y));
    y = __builtin_fmaf(b, t.x, a * t.y);
}

// Work items of one head: first the rotated part (HALF: VEC pairs, two accesses; interleaved: one
// access of VEC elements, or one pair when VEC = 1), then the copied rest, VEC elements each.
template <bool F32, int VEC, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(ikbo_rope_args a, int tokens_per_block) {
    extern __shared__ float2 cs[];   // [tokens][rot_dim / 2]: factor * (cos, sin)
    constexpr int SIZE = F32 ? 4 : 2;
    const int half = a.rot_dim / 2, tid = (int)threadIdx.x;
    const long long t0 = (long long)blockIdx.x * tokens_per_block;
    const int nt = (int)min((long long)tokens_per_block, a.T - t0);
    for (int x = tid; x < nt * half; x += kThreads) {
        const int tt = x / half, i = x - tt * half;
        const double turns = (double)a.positions[t0 + tt] * (a.freq[i] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[x] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
    }
    __syncthreads();
    constexpr int RSTEP = HALF || VEC > 1 ? VEC : 2;                  // elements of the rotated part per item
    const int n_rot = (HALF ? half : a.rot_dim) / RSTEP;
    const int rest = a.head_dim - a.rot_dim;
    const int per_head = n_rot + rest / VEC;
    const int heads = a.H_q + a.H_k, per_token = heads * per_head;
    for (int x = tid; x < nt * per_token; x += kThreads) {
        const int tt = x / per_token, y = x - tt * per_token;
        int h = y / per_head;
        const int c = y - h * per_head;
        const bool is_q = h < a.H_q;
        if (!is_q) h -= a.H_q;
        const char *in = static_cast<const char *>(is_q ? a.q : a.k) +
                         SIZE * ((t0 + tt) * (is_q ? a.q_token : a.k_token) + h * (is_q ? a.q_head : a.k_head));
        char *out = static_cast<char *>(is_q ? a.q_out : a.k_out) +
                    SIZE * ((t0 + tt) * (is_q ? a.q_out_token : a.k_out_token) + h * (is_q ? a.q_out_head : a.k_out_head));
        const float2 *w = cs + tt * half;
        if (c >= n_rot) {
            const int d = a.rot_dim + (c - n_rot) * VEC;
            Vec<F32, VEC> v;
            v.load(in + SIZE * d);
            v.store(out + SIZE * d);
        } else if constexpr (HALF) {
            const int d = c * VEC;
            Vec<F32, VEC> u, v;
            u.load(in + SIZE * d);
            v.load(in + SIZE * (d + half));
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 t = w[d + e];
                const float x0 = u.x[e], x1 = v.x[e];
                turn(x0, x1, t, u.x[e], v.x[e]);
            }
            u.store(out + SIZE * d);
            v.store(out + SIZE * (d + half));
        } else if constexpr (VEC > 1) {
            const int d = c * VEC;
            Vec<F32, VEC> v;
            v.load(in + SIZE * d);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 t = w[(d + e) / 2];
                const float x0 = v.x[e], x1 = v.x[e + 1];
                turn(x0, x1, t, v.x[e], v.x[e + 1]);
            }
            v.store(out + SIZE * d);
        } else {
            const int d = 2 * c;
            Vec<F32, 1> u, v;
            u.load(in + SIZE * d);
            v.load(in + SIZE * (d + 1));
            const float2 t = w[c];
            const float x0 = u.x[0], x1 = v.x[0];
            turn(x0, x1, t, u.x[0], v.x[0]);
            u.store(out + SIZE * d);
            v.store(out + SIZE * (d + 1));
        }
    }
}

template <bool F32, int VEC, bool HALF>
hipError_t launch(const ikbo_rope_args &a, hipStream_t s) {
    // Several tokens share a block once there are enough blocks for the chip without it: their
    // sines then fill the block's threads.
    const int half = a.rot_dim / 2;
    int tpb = std::max(1, std::min(kThreads / half, a.T / 2048));
    // A launch counts its threads in 32 bits (more are dropped without an error): 2^23 blocks at a time.
    const long long most = (1ll << 23) * tpb;
    for (long long t = 0; t < a.T; t += most) {
        ikbo_rope_args part = a;
        constexpr int SIZE = F32 ? 4 : 2;
        part.T = (int)std::min(most, a.T - t);
        part.positions += t;
        part.q = beyond(a.q, t * a.q_token, SIZE);
        part.k = beyond(a.k, t * a.k_token, SIZE);
        part.q_out = beyond(a.q_out, t * a.q_out_token, SIZE);
        part.k_out = beyond(a.k_out, t * a.k_out_token, SIZE);
        hipLaunchKernelGGL((rope_kernel<F32, VEC, HALF>), dim3((unsigned)((part.T + (long long)tpb - 1) / tpb)), dim3(kThreads),
                           (size_t)tpb * half * sizeof(float2), s, part, tpb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool F32, bool HALF>
hipError_t launch_vec(const ikbo_rope_args &a, hipStream_t s) {
    constexpr int VEC = F32 ? 4 : 8;
    auto whole = [](long long x) { return x % VEC == 0; };
    auto base = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool k_ok = a.H_k == 0 || (base(a.k) && base(a.k_out) && whole(a.k_token) && whole(a.k_head) &&
                                     whole(a.k_out_token) && whole(a.k_out_head));
    const bool q_ok = a.H_q == 0 || (base(a.q) && base(a.q_out) && whole(a.q_token) && whole(a.q_head) &&
                                     whole(a.q_out_token) && whole(a.q_out_head));
    const bool dims = whole(HALF ? a.rot_dim / 2 : a.rot_dim) && whole(a.head_dim);
    return q_ok && k_ok && dims ? launch<F32, VEC, HALF>(a, s) : launch<F32, 1, HALF>(a, s);
}

}  // namespace

hipError_t launch_rope(const ikbo_rope_args &a, hipStream_t s) {
    const bool half = a.layout == IKBO_ROPE_HALF;
    if (a.dtype == IKBO_DTYPE_F32) return half ? launch_vec<true, true>(a, s) : launch_vec<true, false>(a, s);
    return half ? launch_vec<false, true>(a, s) : launch_vec<false, false>(a, s);
}

}  // namespace ikbo
