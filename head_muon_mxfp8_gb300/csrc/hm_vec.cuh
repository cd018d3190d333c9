// Arithmetic on two floats at a time (f32x2), and W neighbouring elements of a bf16 or fp32 row as raw 32-bit words: loaded and
// stored in the widest pieces, up to 16 bytes, that W elements make.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace hm {

__device__ __forceinline__ uint64_t pack2(float2 v) {
    return static_cast<uint64_t>(__float_as_uint(v.x)) | (static_cast<uint64_t>(__float_as_uint(v.y)) << 32);
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
    return unpack2(r);
}
__device__ __forceinline__ float2 both2(float v) { return make_float2(v, v); }

template <bool F32, int W>
struct RowVec {
    static constexpr int kBytes = W * (F32 ? 4 : 2);
    static constexpr int N = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = 0u;
    }
    // whole and aligned to min(kBytes, 16)
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const char* p = static_cast<const char*>(base) + at * (F32 ? 4 : 2);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + k);
                w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = __ldcs(reinterpret_cast<const uint16_t*>(p));
        }
    }
    // the first `count`, one by one, the others zero
    __device__ __forceinline__ void load_some(const void* base, int64_t at, int count) {
        clear();
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (k < count) {
                if (F32) w[F32 ? k : 0] = __ldcs(static_cast<const uint32_t*>(base) + at + k);
                else w[k / 2 % N] |= static_cast<uint32_t>(__ldcs(static_cast<const uint16_t*>(base) + at + k)) << (16 * (k & 1));
            }
    }
    __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
        for (int k = 0; k < W; ++k)
            v[k] = F32 ? __uint_as_float(w[F32 ? k : 0])
                       : __uint_as_float(k & 1 ? w[k / 2 % N] & 0xFFFF0000u : w[k / 2 % N] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[W]) {
        if constexpr (F32) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = __float_as_uint(v[k]);
        } else if constexpr (W == 1) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at) const {
        char* p = static_cast<char*>(base) + at * (F32 ? 4 : 2);
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k)
                reinterpret_cast<uint4*>(p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        }
    }
    __device__ __forceinline__ void store_some(void* base, int64_t at, int count) const {
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (k < count) {
                if (F32) static_cast<uint32_t*>(base)[at + k] = w[F32 ? k : 0];
                else static_cast<uint16_t*>(base)[at + k] = static_cast<uint16_t>(w[k / 2 % N] >> (16 * (k & 1)));
            }
    }
    static __device__ __forceinline__ void put(void* base, int64_t at, const float (&v)[W]) {
        RowVec r;
        r.set(v);
        r.store(base, at);
    }
};

}  // namespace hm
