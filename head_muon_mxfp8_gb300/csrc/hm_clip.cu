// Global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum g^2), coef = min(1, max_norm / (norm + eps)), g <- g coef.
//
// The tensors' table travels in the kernel's parameters.  A tensor is cut into
// chunks of 4096 16-byte vectors from its first 16-byte boundary; its first
// chunk also takes the elements before that boundary and its last one those
// after the last whole vector, so any element alignment runs on vector loads.
// A thread adds the squares of one chunk's 16 vectors in fp32 and carries its
// sum from chunk to chunk in double; CTA sums are doubles too, added in a fixed
// order.  Two launches: the norm pass, and a pass that adds the CTA sums (every CTA
// the same way) and scales.  The second pass has to read the gradient again; it
// walks the chunks backwards, and the norm pass marks all but the last ones
// (as much as half the L2 holds) evict-first, so those come from the L2.
// A thread's fp32 sum that overflowed or may have underflowed (squares
// leave fp32 for |g| > 2^63 or < 2^-63) is formed again in double.
#include "hm_internal.h"
#include "hm_ops.h"

#include <cuda_bf16.h>

#include <algorithm>

namespace hm {

namespace {

constexpr int kClipThreads = 256;
constexpr int kChunkVecs = 4096;  // 16-byte vectors per chunk, 16 per thread
constexpr int kClipUnroll = 8;

struct Place {   // a chunk of a tensor
    int64_t v0;      // its first vector
    int nv;          // its vectors
    int64_t head;    // elements before the first vector
    int64_t tail0;   // first element after the last vector
    bool first, last;
};

__device__ __forceinline__ int find_tensor(const ClipArgs& a, int chunk) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ Place place_of(const ClipTensor& t, int chunk) {
    const int es = t.f32 ? 4 : 2, ve = 16 / es;
    Place c;
    c.head = min(t.n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(t.src) & 15)) & 15) / es));
    const int64_t nv = (t.n - c.head) / ve;
    c.tail0 = c.head + nv * ve;
    c.v0 = static_cast<int64_t>(chunk - t.first) * kChunkVecs;
    c.nv = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kChunkVecs), nv - c.v0)));
    c.first = chunk == t.first;
    c.last = c.v0 + kChunkVecs >= nv;
    return c;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float one_value(const ClipTensor& t, int64_t e) {
    return t.f32 ? static_cast<const float*>(t.src)[e]
                 : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(t.src)[e]) << 16);
}

// squares of one vector; bits collects the magnitudes (0 when every value is 0)
template <bool F32>
__device__ __forceinline__ void add_squares(const uint4& x, float& s, uint32_t& bits) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (F32) {
            const float v = __uint_as_float(w[k]);
            s = fmaf(v, v, s);
            bits |= w[k] & 0x7FFFFFFFu;
        } else {
            const float a = bf16_lo(w[k]), b = bf16_hi(w[k]);
            s = fmaf(a, a, s);
            s = fmaf(b, b, s);
            bits |= w[k] & 0x7FFF7FFFu;
        }
    }
}

template <bool F32>
__device__ __noinline__ double squares_in_double(const uint4* src, int nv) {
    double s = 0.0;
    for (int i = threadIdx.x; i < nv; i += kClipThreads) {
        const uint4 x = src[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        for (int k = 0; k < 4; ++k) {
            if (F32) {
                const double v = __uint_as_float(w[k]);
                s += v * v;
            } else {
                const double a = bf16_lo(w[k]), b = bf16_hi(w[k]);
                s += a * a + b * b;
            }
        }
    }
    return s;
}

template <bool F32>
__device__ __forceinline__ double chunk_squares(const uint4* src, int nv, bool keep) {
    float s = 0.f;
    uint32_t bits = 0;
    for (int i0 = threadIdx.x; i0 < nv; i0 += kClipUnroll * kClipThreads) {
        uint4 x[kClipUnroll];
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) {
            const int i = i0 + u * kClipThreads;
            x[u] = i >= nv ? make_uint4(0u, 0u, 0u, 0u) : keep ? __ldcg(src + i) : __ldcs(src + i);
        }
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) add_squares<F32>(x[u], s, bits);
    }
    // 2^-90: squares lost to underflow are then below 2^-29 of the sum
    if (bits && !(s >= 0x1p-90f && s <= 3.4028234664e38f)) return squares_in_double<F32>(src, nv);
    return s;
}

// Sum over the CTA in a fixed order, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kClipThreads / 32; ++k) t += red[k];
    return t;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipArgs a) {
    double sum = 0.0;
    for (int ch = blockIdx.x; ch < a.chunks; ch += gridDim.x) {
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        const Place c = place_of(t, ch);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(t.src) + c.head * (t.f32 ? 4 : 2)) + c.v0;
        const bool keep = ch >= a.keep_from;
        sum += t.f32 ? chunk_squares<true>(src, c.nv, keep) : chunk_squares<false>(src, c.nv, keep);
        if (c.first && threadIdx.x < c.head) {
            const double v = one_value(t, threadIdx.x);
            sum += v * v;
        }
        if (c.last && c.tail0 + threadIdx.x < t.n) {
            const double v = one_value(t, c.tail0 + threadIdx.x);
            sum += v * v;
        }
    }
    const double total = block_sum(sum);
    if (threadIdx.x == 0) a.partials[a.part0 + blockIdx.x] = total;
}

__device__ __forceinline__ void store_value(const ClipTensor& t, int64_t e, float v) {
    if (t.f32) static_cast<float*>(t.dst)[e] = v;
    else static_cast<uint16_t*>(t.dst)[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, float c) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(bf16_lo(w) * c, bf16_hi(w) * c);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipArgs a) {
    __shared__ float s_coef;
    double sum = 0.0;
    for (int k = threadIdx.x; k < a.parts; k += kClipThreads) sum += a.partials[k];
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const float norm = static_cast<float>(sqrt(sum));
        const float c = a.max_norm / (norm + a.eps);
        s_coef = c >= 1.f ? 1.f : c;  // a NaN stays
        if (blockIdx.x == 0 && a.part0 == 0) {
            a.stats[0] = norm;
            a.stats[1] = s_coef;
        }
    }
    __syncthreads();
    const float coef = s_coef;
    for (int k = blockIdx.x; k < a.chunks; k += gridDim.x) {
        const int ch = a.chunks - 1 - k;  // the chunks the norm pass read last are still in the L2
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        if (!t.dst || (t.dst == t.src && coef == 1.f)) continue;
        const Place c = place_of(t, ch);
        const int es = t.f32 ? 4 : 2;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(t.src) + c.head * es) + c.v0;
        char* out = static_cast<char*>(t.dst) + c.head * es + c.v0 * 16;
        const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        for (int i0 = threadIdx.x; i0 < c.nv; i0 += kClipUnroll * kClipThreads) {
            uint4 x[kClipUnroll];
#pragma unroll
            for (int u = 0; u < kClipUnroll; ++u) {
                const int i = i0 + u * kClipThreads;
                if (i < c.nv) x[u] = __ldcs(src + i);
            }
#pragma unroll
            for (int u = 0; u < kClipUnroll; ++u) {
                const int i = i0 + u * kClipThreads;
                if (i >= c.nv) continue;
                uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = t.f32 ? __float_as_uint(__uint_as_float(w[k]) * coef) : scale_bf16x2(w[k], coef);
                if (vec) {
                    __stcs(reinterpret_cast<uint4*>(out) + i, make_uint4(w[0], w[1], w[2], w[3]));
                } else if (t.f32) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) reinterpret_cast<uint32_t*>(out)[i * 4 + k] = w[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        reinterpret_cast<uint16_t*>(out)[i * 8 + k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
                }
            }
        }
        if (c.first && threadIdx.x < c.head) store_value(t, threadIdx.x, one_value(t, threadIdx.x) * coef);
        if (c.last && c.tail0 + threadIdx.x < t.n)
            store_value(t, c.tail0 + threadIdx.x, one_value(t, c.tail0 + threadIdx.x) * coef);
    }
}

}  // namespace

int clip_chunks(const void* src, int64_t n, int f32) {
    const int es = f32 ? 4 : 2;
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / es;
    if (head > n) head = n;
    const int64_t nv = (n - head) / (16 / es);
    return static_cast<int>(nv <= kChunkVecs ? 1 : (nv + kChunkVecs - 1) / kChunkVecs);
}

int clip_parts(int chunks) {
    const int most = 4 * device_sm_count();
    return chunks < most ? chunks : most;
}

cudaError_t launch_clip_norm(ClipArgs& a, cudaStream_t st) {
    a.keep_from = static_cast<int32_t>(std::max<int64_t>(0, a.chunks - device_l2_bytes() / 2 / (kChunkVecs * 16)));
    note_launch();
    clip_norm_kernel<<<clip_parts(a.chunks), kClipThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_clip_scale(const ClipArgs& a, cudaStream_t st) {
    note_launch();
    clip_scale_kernel<<<a.chunks ? clip_parts(a.chunks) : 1, kClipThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace hm
