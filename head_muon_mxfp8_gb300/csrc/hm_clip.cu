// Global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum g^2), coef = min(1, max_norm / (norm + eps)), g <- g coef.
//
// The tensors' table travels in the kernel's parameters.  A tensor is cut into
// chunks of 4096 16-byte vectors from its first 16-byte boundary; its first
// chunk also takes the elements before that boundary and its last one those
// after the last whole vector, so any element alignment runs on vector loads.
// A thread adds the squares of one chunk's 16 vectors in fp32 and carries its
// sum from chunk to chunk in double; a warp's 32 sums are joined in fp32 (five
// roundings) where all are well inside its range, else in double; the warps' and
// CTAs' sums are doubles.  All in a fixed order.  Two launches (one for little data, at the end): the norm pass, and a pass that
// adds the CTA sums (every CTA the same way) and scales.  The second pass has to read the gradient again; it
// walks the chunks backwards, and the norm pass marks all but the last ones
// (as much as half the L2 holds) evict-first, so those come from the L2.
// A thread's fp32 sum that overflowed or may have underflowed (squares
// leave fp32 for |g| > 2^63 or < 2^-63) is formed again in double.
// Memory-bound: 131 M fp32 elements in 48 tensors take 252 us out of place, the same
// in bf16 120.
#include "hm_internal.h"
#include "hm_ops.h"
#include "hm_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace hm {

namespace {

constexpr int kClipThreads = 256;
constexpr int kChunkVecs = kClipChunkVecs;  // 16 per thread
constexpr int kClipUnroll = 8;

struct Place {   // a chunk of a tensor
    int64_t v0;      // its first vector
    int nv;          // its vectors
    int64_t head;    // elements before the first vector
    int64_t tail0;   // first element after the last vector
    bool first, last;
};

template <int CAP>
__device__ __forceinline__ int find_tensor(const ClipArgs<CAP>& a, int chunk) {
    int lo = 0, hi = a.h.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int VECS>
__device__ __forceinline__ Place place_of(const ClipTensor& t, int chunk) {
    const int es = t.f32 ? 4 : 2, ve = 16 / es;
    Place c;
    c.head = min(t.n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(t.src) & 15)) & 15) / es));
    const int64_t nv = (t.n - c.head) / ve;
    c.tail0 = c.head + nv * ve;
    c.v0 = static_cast<int64_t>(chunk - t.first) * VECS;
    c.nv = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(VECS), nv - c.v0)));
    c.first = chunk == t.first;
    c.last = c.v0 + VECS >= nv;
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

// The same in double.
__device__ __noinline__ double squares_in_double(uint4 x, int f32) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    double s = 0.0;
    for (int k = 0; k < 4; ++k) {
        const double a = f32 ? __uint_as_float(w[k]) : bf16_lo(w[k]), b = f32 ? 0.f : bf16_hi(w[k]);
        s += a * a + b * b;
    }
    return s;
}

// Whether fp32 holds a sum of squares s whose terms' magnitudes are in bits:
// 2^-90, so that squares lost to underflow are below 2^-29 of the sum.
__device__ __forceinline__ bool in_range(float s, uint32_t bits) {
    return !bits || (s >= 0x1p-90f && s <= 3.4028234664e38f);
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
    if (in_range(s, bits)) return s;
    double d = 0.0;
    for (int i = threadIdx.x; i < nv; i += kClipThreads) d += squares_in_double(src[i], F32);
    return d;
}

// Sum over the warp in a fixed order: in fp32 (five additions) where every lane's
// value is well inside its range, since 32 lanes adding doubles take 16 clocks of the
// SM's double units each time; else in double.
__device__ __forceinline__ double warp_sum(double v) {
    float f = static_cast<float>(v);
    if (__all_sync(0xffffffffu, f == 0.f ? v == 0.0 : f >= 0x1p-100f && f <= 0x1p100f)) {
#pragma unroll
        for (int o = 16; o; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
        return f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the CTA in a fixed order, in thread 0.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[THREADS / 32];
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x < 32) {
        t = threadIdx.x < THREADS / 32 ? red[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return t;
}

__device__ __forceinline__ const uint4* place_src(const ClipTensor& t, const Place& c) {
    return reinterpret_cast<const uint4*>(static_cast<const char*>(t.src) + c.head * (t.f32 ? 4 : 2)) + c.v0;
}

// Squares of the elements of a chunk before its first and after its last vector.
__device__ __forceinline__ double end_squares(const ClipTensor& t, const Place& c, int tid) {
    double sum = 0.0;
    if (c.first && tid < c.head) {
        const double v = one_value(t, tid);
        sum += v * v;
    }
    if (c.last && c.tail0 + tid < t.n) {
        const double v = one_value(t, c.tail0 + tid);
        sum += v * v;
    }
    return sum;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipArgs<kClipTensors> a) {
    double sum = 0.0;
    wait_for_earlier_kernels();
    for (int ch = blockIdx.x; ch < a.h.chunks; ch += gridDim.x) {
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        const Place c = place_of<kChunkVecs>(t, ch);
        const bool keep = ch >= a.h.keep_from;
        sum += t.f32 ? chunk_squares<true>(place_src(t, c), c.nv, keep) : chunk_squares<false>(place_src(t, c), c.nv, keep);
        sum += end_squares(t, c, threadIdx.x);
    }
    const double total = block_sum<kClipThreads>(sum);
    if (threadIdx.x == 0) a.h.partials[a.h.part0 + blockIdx.x] = total;
}

__device__ __forceinline__ void store_value(const ClipTensor& t, int64_t e, float v) {
    if (t.f32) static_cast<float*>(t.dst)[e] = v;
    else static_cast<uint16_t*>(t.dst)[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, float c) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(bf16_lo(w) * c, bf16_hi(w) * c);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// coef from the sum of squares; writes stats if asked.
__device__ __forceinline__ float coefficient(const ClipHead& h, double sum, bool write) {
    // one rounding of the sum and the root's in fp32 wherever it holds the sum
    const float f = static_cast<float>(sum);
    const float norm = f >= 0x1p-100f && f <= 0x1p100f ? sqrtf(f) : static_cast<float>(sqrt(sum));
    // a NaN norm compares false and stays; an infinite max_norm never clips
    const float coef = norm + h.eps <= h.max_norm ? 1.f : h.max_norm / (norm + h.eps);
    if (write) {
        h.stats[0] = norm;
        h.stats[1] = coef;
    }
    return coef;
}

// One vector times coef to element-aligned (vec: 16-byte aligned) memory.
__device__ __forceinline__ void store_scaled(const ClipTensor& t, const uint4& x, float coef, char* out, bool vec) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = t.f32 ? __float_as_uint(__uint_as_float(w[k]) * coef) : scale_bf16x2(w[k], coef);
    if (vec) {
        __stcs(reinterpret_cast<uint4*>(out), make_uint4(w[0], w[1], w[2], w[3]));
    } else if (t.f32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) reinterpret_cast<uint32_t*>(out)[k] = w[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) reinterpret_cast<uint16_t*>(out)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
}

__device__ __forceinline__ char* place_dst(const ClipTensor& t, const Place& c) {
    return static_cast<char*>(t.dst) + c.head * (t.f32 ? 4 : 2) + c.v0 * 16;
}

// The elements of a chunk before its first and after its last vector.
__device__ __forceinline__ void scale_ends(const ClipTensor& t, const Place& c, float coef, int tid) {
    if (c.first && tid < c.head) store_value(t, tid, one_value(t, tid) * coef);
    if (c.last && c.tail0 + tid < t.n) store_value(t, c.tail0 + tid, one_value(t, c.tail0 + tid) * coef);
}

__device__ __forceinline__ void scale_place(const ClipTensor& t, const Place& c, float coef) {
    const uint4* src = place_src(t, c);
    char* out = place_dst(t, c);
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
            if (i < c.nv) store_scaled(t, x[u], coef, out + static_cast<int64_t>(i) * 16, vec);
        }
    }
    scale_ends(t, c, coef, threadIdx.x);
}

__device__ __forceinline__ bool to_scale(const ClipTensor& t, float coef) {
    return t.dst && !(t.dst == t.src && coef == 1.f);
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipArgs<kClipTensors> a) {
    __shared__ float s_coef;
    double sum = 0.0;
    wait_for_earlier_kernels();
    if (threadIdx.x < 32) {  // one warp: the SM's double units would hold up four CTAs' worth of more
        for (int k = threadIdx.x; k < a.h.parts; k += 32) sum += a.h.partials[k];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (threadIdx.x == 0) s_coef = coefficient(a.h, sum, blockIdx.x == 0 && a.h.part0 == 0);
    __syncthreads();
    const float coef = s_coef;
    for (int k = blockIdx.x; k < a.h.chunks; k += gridDim.x) {
        const int ch = a.h.chunks - 1 - k;  // the chunks the norm pass read last are still in the L2
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        if (to_scale(t, coef)) scale_place(t, place_of<kChunkVecs>(t, ch), coef);
    }
}

// Little data in few tensors: one cluster of 8 CTAs does both passes, the CTA
// sums exchanged through distributed shared memory -- one launch instead of two
// and a table of 0.5 KB instead of 8 (200,000 fp32 elements in 5 tensors: 12.3 us a call
// with two launches, 10.2 with one when both were measured; 7.9 since the launch
// overlaps the kernel before).
// A CTA is four groups of kClipThreads; a group holds its two chunks in registers
// from the first pass to the second.
constexpr int kFewCtas = 8;
constexpr int kFewThreads = 4 * kClipThreads;
constexpr int kFewGroups = kFewCtas * kFewThreads / kClipThreads;
constexpr int kFewPerGroup = kClipFewChunks / kFewGroups;
constexpr int kFewVecs = kClipFewChunkVecs / kClipThreads;  // of a chunk per thread
__global__ void __cluster_dims__(kFewCtas, 1, 1) __launch_bounds__(kFewThreads)
    clip_few_kernel(const __grid_constant__ ClipArgs<kClipFew> a) {
    __shared__ double s_part;
    __shared__ float s_coef;
    wait_for_earlier_kernels();
    const int tid = threadIdx.x % kClipThreads;
    const int group = blockIdx.x + kFewCtas * (threadIdx.x / kClipThreads);
    uint4 x[kFewPerGroup][kFewVecs];
#pragma unroll
    for (int g = 0; g < kFewPerGroup; ++g) {
        const int ch = group + g * kFewGroups;
#pragma unroll
        for (int u = 0; u < kFewVecs; ++u) x[g][u] = make_uint4(0u, 0u, 0u, 0u);
        if (ch < a.h.chunks) {
            const ClipTensor& t = a.t[find_tensor(a, ch)];
            const Place c = place_of<kClipFewChunkVecs>(t, ch);
            const uint4* src = place_src(t, c);
#pragma unroll
            for (int u = 0; u < kFewVecs; ++u)
                if (tid + u * kClipThreads < c.nv) x[g][u] = src[tid + u * kClipThreads];
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int g = 0; g < kFewPerGroup; ++g) {
        const int ch = group + g * kFewGroups;
        if (ch >= a.h.chunks) continue;
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        float s = 0.f;
        uint32_t bits = 0;
#pragma unroll
        for (int u = 0; u < kFewVecs; ++u) {
            if (t.f32) add_squares<true>(x[g][u], s, bits);
            else add_squares<false>(x[g][u], s, bits);
        }
        if (in_range(s, bits)) sum += s;
        else
#pragma unroll
            for (int u = 0; u < kFewVecs; ++u) sum += squares_in_double(x[g][u], t.f32);
        sum += end_squares(t, place_of<kClipFewChunkVecs>(t, ch), tid);
    }
    sum = block_sum<kFewThreads>(sum);
    if (threadIdx.x == 0) s_part = sum;
    __syncwarp();
    cluster_sync_all();
    if (threadIdx.x == 0) {
        double part[kFewCtas];
#pragma unroll
        for (int k = 0; k < kFewCtas; ++k)
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(part[k]) : "r"(mapa_shared(smem_u32(&s_part), k)) : "memory");
#pragma unroll
        for (int w = kFewCtas / 2; w; w >>= 1)
#pragma unroll
            for (int k = 0; k < w; ++k) part[k] += part[k + w];
        const double total = part[0];
        s_coef = coefficient(a.h, total, blockIdx.x == 0);
    }
    __syncthreads();
    cluster_arrive_relaxed();  // this CTA has read its peers' sums
    const float coef = s_coef;
#pragma unroll
    for (int g = 0; g < kFewPerGroup; ++g) {
        const int ch = group + g * kFewGroups;
        if (ch >= a.h.chunks) continue;
        const ClipTensor& t = a.t[find_tensor(a, ch)];
        if (!to_scale(t, coef)) continue;
        const Place c = place_of<kClipFewChunkVecs>(t, ch);
        char* out = place_dst(t, c);
        const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
        for (int u = 0; u < kFewVecs; ++u) {
            const int i = tid + u * kClipThreads;
            if (i < c.nv) store_scaled(t, x[g][u], coef, out + i * 16, vec);
        }
        scale_ends(t, c, coef, tid);
    }
    __syncwarp();
    cluster_wait();  // a CTA's sum stays until its peers have read it
}

}  // namespace

int clip_chunks(const void* src, int64_t n, int f32, int vecs) {
    const int es = f32 ? 4 : 2;
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / es;
    if (head > n) head = n;
    const int64_t nv = (n - head) / (16 / es);
    return static_cast<int>(nv <= vecs ? 1 : (nv + vecs - 1) / vecs);
}

int clip_parts(int chunks) {
    const int most = 4 * device_sm_count();
    return chunks < most ? chunks : most;
}

cudaError_t launch_clip_norm(ClipArgs<kClipTensors>& a, cudaStream_t st) {
    a.h.keep_from = static_cast<int32_t>(std::max<int64_t>(0, a.h.chunks - device_l2_bytes() / 2 / (kChunkVecs * 16)));
    note_launch();
    return launch_early(clip_norm_kernel, clip_parts(a.h.chunks), kClipThreads, 0, st, a);
}

cudaError_t launch_clip_scale(const ClipArgs<kClipTensors>& a, cudaStream_t st) {
    note_launch();
    return launch_early(clip_scale_kernel, clip_parts(a.h.chunks), kClipThreads, 0, st, a);
}

cudaError_t launch_clip_few(const ClipArgs<kClipFew>& a, cudaStream_t st) {
    note_launch();
    return launch_early(clip_few_kernel, kFewCtas, kFewThreads, 0, st, a);
}

}  // namespace hm
