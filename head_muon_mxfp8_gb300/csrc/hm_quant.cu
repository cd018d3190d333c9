// MXFP8 quantization of activations, gradients and weights along either axis.
//
// y = x * row * col (fp32); per block of 32 (or 128) elements along an axis,
// e = clamp(floor(log2 amax) - 8, -127, 127), codes E4M3_RNE(y 2^-e), scale
// byte e + 127 -- G's rule (hm_mx_device.cuh).  x is read once for both axes:
// the gradient products of a linear layer contract along the tokens, so they
// need the transposed operand of what the forward product uses.
//
// A CTA takes a 128 x 128 tile: the tile's scales are then one 512-byte tile of
// either scale layout.  Memory-bound: bf16 x with both outputs moves
// 2 + 2 (1 + 1/32) bytes per element.
// 8192 x 15360 bf16 to both outputs takes 80 us (6.4 TB/s, 0.94 of the measured
// copy rate); a 14336 x 4096 fp32 weight to its transpose 63 us (4.7 TB/s), where
// registers for the loads leave two CTAs per SM (a third CTA's spill: 92 us;
// 512 threads per CTA: 66 us); 8192 x 5120 bf16 with both factors, the fp32 tile too,
// 35.2 us to its transpose (3.6 TB/s) and 45.8 both ways.  With the sums of the columns
// (mxfp8_quantize_bias) 8192 x 20480 bf16 both ways takes 111 us, 106 without; the sums come
// from the tile in shared memory, a row of the workspace per row tile, added by a second
// launch (none for up to 128 rows).
#include "hm_internal.h"
#include "hm_mx_device.cuh"
#include "hm_ops.h"
#include "hm_ptx.cuh"
#include "hm_vec.cuh"

namespace hm {

namespace {

constexpr int kQThreads = 256;
constexpr int kQTile = 128;

// 16 elements of a row of x as loaded, those from `left` on being zero.
template <bool F32>
struct Raw16 {
    static constexpr int N = F32 ? 4 : 2;
    uint4 w[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void load(const void* x, int64_t at, int left, bool vec) {
        if (vec && left == 16) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (F32 ? 4 : 2));
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = __ldcs(p + k);
            return;
        }
        uint32_t h[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            h[k] = k >= left ? 0u
                   : F32     ? static_cast<const uint32_t*>(x)[at + k]
                             : static_cast<uint32_t>(static_cast<const uint16_t*>(x)[at + k]);
#pragma unroll
        for (int k = 0; k < N; ++k)
            w[k] = F32 ? make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3])
                       : make_uint4(h[(8 * k) & 15] | (h[(8 * k + 1) & 15] << 16), h[(8 * k + 2) & 15] | (h[(8 * k + 3) & 15] << 16),
                                    h[(8 * k + 4) & 15] | (h[(8 * k + 5) & 15] << 16), h[(8 * k + 6) & 15] | (h[(8 * k + 7) & 15] << 16));
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    v[(4 * k + j) & 15] = __uint_as_float(u[j]);
                } else {
                    v[(8 * k + 2 * j) & 15] = __uint_as_float(u[j] << 16);
                    v[(8 * k + 2 * j + 1) & 15] = __uint_as_float(u[j] & 0xFFFF0000u);
                }
            }
        }
    }
};

// Where the fp32 tile keeps 16-byte piece k of a row: no bank twice, neither for the
// row phase's lanes (64 bytes apart) nor for a column's readers (the exchange
// stays inside 128 bytes).
__device__ __forceinline__ int swizzled(int k) { return k ^ (k >> 3); }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float sc) {
    return cvt_e4m3x2(a * sc, b * sc) | (static_cast<uint32_t>(cvt_e4m3x2(c * sc, d * sc)) << 16);
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Elementwise max of the magnitudes of two bf16 pairs, up to the sign bits (a
// NaN is left out, as by fmaxf).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
// 2^-e as bf16 for a scale's byte, and the product with it: a power of two, so
// exact wherever the result is not far below the smallest code.
__device__ __forceinline__ uint32_t inv_of_byte_bf16(int byte) { return static_cast<uint32_t>(254 - byte) << 7; }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}
__device__ __forceinline__ uint32_t join(uint16_t lo, uint16_t hi) {
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// qt's tile leaves through shared memory, [128 columns][128 codes], so that a
// warp stores four whole lines: stored straight from the column phase, 32 bytes
// of 32 rows at a time, the transposed output took 36 of 102 us as two 16-byte
// halves per sector and 25 as one sector per lane.  16-byte piece k of column c
// sits at piece k ^ key(c): no bank twice, whether lanes hold consecutive
// columns or every other one.
__device__ __forceinline__ int stage_key(int c) { return (c + (c >> 3)) & 7; }
__device__ __forceinline__ void stage_codes32(uint4* stage, int c, int b, const uint32_t (&x)[8]) {
    const int k = stage_key(c);
    stage[c * 8 + ((2 * b) ^ k)] = make_uint4(x[0], x[1], x[2], x[3]);
    stage[c * 8 + ((2 * b + 1) ^ k)] = make_uint4(x[4], x[5], x[6], x[7]);
}

// The block's scale byte from this lane's amax over 16 of its columns.
__device__ __forceinline__ int row_scale(float amax, int block) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (block == 128) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
    }
    return mx_scale_byte(amax);
}

// The sums of the tile's columns over each of its four 32-row blocks.
template <bool PACKED>
__device__ __forceinline__ void sum_columns(const uint32_t* tile, float (*sum_col)[kQTile]) {
    if constexpr (PACKED) {
        const int cp = threadIdx.x & 63, b = threadIdx.x >> 6;
        float2 sum = both2(0.f);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const uint32_t w = tile[(b * 32 + k) * (kQTile / 2) + cp];
            sum = add2(sum, make_float2(lo_f32(w), hi_f32(w)));
        }
        sum_col[b][2 * cp] = sum.x;
        sum_col[b][2 * cp + 1] = sum.y;
    } else {
        const int c = threadIdx.x & 127;
        const float* col = reinterpret_cast<const float*>(tile) + 4 * swizzled(c >> 2) + (c & 3);
        for (int b = threadIdx.x >> 7; b < 4; b += kQThreads / 128) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) s += col[(b * 32 + k) * kQTile];
            sum_col[b][c] = s;
        }
    }
}
// Those, added: a row of the workspace, or dbias itself where this is the only row tile.
__device__ __forceinline__ void store_sums(const QuantArgs& p, const float (*sum_col)[kQTile], int64_t c0, int64_t rt) {
    const int c = threadIdx.x;
    if (c >= kQTile || c0 + c >= p.cols) return;
    float* to = p.sums + rt * p.cols + c0 + c;
    const float s = (sum_col[0][c] + sum_col[1][c]) + (sum_col[2][c] + sum_col[3][c]);
    *to = p.sums_add ? *to + s : s;
}

// Row phase: 8 lanes hold a row of the tile, 16 columns each (two lanes per
// block of 32), a warp 16 rows in four steps whose loads are all issued before
// the first is used.  16 columns per lane rather than 8: the work per block
// (exponent, scale, addresses) is shared by more of them; at 8 the kernel
// issued 20 instructions per element and the issue slots bounded it.
// The tile, in two forms:
//   PACKED (bf16 x, no factors): y is x, so the tile stays in bf16 pairs --
//     half the shared memory and half its traffic, and magnitudes are compared
//     two at a time; a thread's column work is a pair of columns x 32 rows.
//   else: y in fp32 (swizzled); a thread's column work is one column x 32 rows.
// SUM: the sums of the tile's columns too, from the tile in shared memory: a thread's
// column work is summed row by row, then the 32-row blocks in order.
template <bool F32, bool PACKED, bool COL, bool SUM>
__global__ void __launch_bounds__(kQThreads, PACKED ? 4 : 2) quantize_kernel(const __grid_constant__ QuantArgs p) {
    constexpr bool TILE = COL || SUM;
    extern __shared__ __align__(16) uint32_t tile[];  // [128][64] bf16 pairs or [128][128] fp32
    __shared__ __align__(16) uint8_t s_row[512];
    __shared__ __align__(16) uint8_t s_col[512];
    __shared__ float amax_col[4][kQTile];
    __shared__ float sum_col[SUM ? 4 : 1][kQTile];
    wait_for_earlier_kernels();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ct = blockIdx.x, rt = blockIdx.y;
    const int64_t r0 = rt * kQTile, c0 = ct * kQTile;
    const int64_t cols32 = (p.cols + 31) / 32 * 32, rows32 = (p.rows + 31) / 32 * 32;
    const int c16 = (lane & 7) * 16;
    const int left = static_cast<int>(min(static_cast<int64_t>(16), max(static_cast<int64_t>(0), p.cols - (c0 + c16))));
    constexpr int kSteps = 128 * 32 / kQThreads / 4;  // rows per warp, four at a time
    const int rl0 = warp * (4 * kSteps) + (lane >> 3);         // this lane's rows: rl0 + 4 i
    const int rows = static_cast<int>(min(static_cast<int64_t>(kQTile), p.rows - r0));  // of the tile
    const bool q_live = p.q && c0 + c16 < cols32;
    const int flip = (lane >> 2) & 1;  // which of its two 16-byte pieces a lane stores first: no bank twice
    uint8_t* qp = p.q + (r0 + rl0) * p.ldq + c0 + c16;

    if constexpr (PACKED) {
        Raw16<false> raw[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            raw[i].clear();
            if (rl0 + 4 * i < rows && left > 0) raw[i].load(p.x, (r0 + rl0 + 4 * i) * p.ldx + c0 + c16, left, p.vec);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int rl = rl0 + 4 * i;
            if (TILE) {
                uint4* t4 = reinterpret_cast<uint4*>(tile + rl * (kQTile / 2) + c16 / 2);
                t4[flip] = flip ? raw[i].w[1] : raw[i].w[0];
                t4[flip ^ 1] = flip ? raw[i].w[0] : raw[i].w[1];
            }
            if (p.q) {
                const uint32_t w[8] = {raw[i].w[0].x, raw[i].w[0].y, raw[i].w[0].z, raw[i].w[0].w,
                                       raw[i].w[1].x, raw[i].w[1].y, raw[i].w[1].z, raw[i].w[1].w};
                uint32_t m = 0u;
#pragma unroll
                for (int k = 0; k < 8; ++k) m = max_abs2(m, w[k]);
                const int byte = row_scale(fmaxf(fabsf(lo_f32(m)), fabsf(hi_f32(m))), p.block);
                const uint32_t sc = inv_of_byte_bf16(byte) * 0x10001u;
                const bool live = q_live && rl < rows;
                if (live) {
                    uint32_t c[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t y0 = mul2(w[2 * k], sc), y1 = mul2(w[2 * k + 1], sc);
                        c[k] = join(cvt_e4m3x2(lo_f32(y0), hi_f32(y0)), cvt_e4m3x2(lo_f32(y1), hi_f32(y1)));
                    }
                    __stcs(reinterpret_cast<uint4*>(qp + 4 * i * p.ldq), make_uint4(c[0], c[1], c[2], c[3]));
                }
                // row rl = rl0 + 4 i of the scale tile: (rl % 32) * 16 + (rl / 32) * 4 + block
                if (!(lane & 1)) s_row[(rl & 31) * 16 + (rl >> 5) * 4 + ((lane & 7) >> 1)] = live ? static_cast<uint8_t>(byte) : 0;
            }
        }
    } else {
        float cm[16];
        if (p.col_vec && left == 16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 f = reinterpret_cast<const float4*>(p.col_mul + c0 + c16)[k];
                cm[4 * k] = f.x; cm[4 * k + 1] = f.y; cm[4 * k + 2] = f.z; cm[4 * k + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) cm[k] = p.col_mul && k < left ? p.col_mul[c0 + c16 + k] : 1.f;
        }
        Raw16<F32> raw[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            raw[j].clear();
            if (rl0 + 4 * j < rows && left > 0) raw[j].load(p.x, (r0 + rl0 + 4 * j) * p.ldx + c0 + c16, left, p.vec);
        }
        {
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const int rl = rl0 + 4 * j;
                float v[16];
                raw[j].get(v);
                if (rl < rows) {  // outside x the zeros stay +0 whatever the factors' signs
                    const float rm = p.row_mul ? p.row_mul[r0 + rl] : 1.f;
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = v[k] * rm * cm[k];
                    if (left < 16)
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = k < left ? v[k] : 0.f;
                }
                if (TILE) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<float4*>(tile + rl * kQTile + 4 * swizzled(c16 / 4 + k)) =
                            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
                if (p.q) {
                    float amax = 0.f;
#pragma unroll
                    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(v[k]));
                    const int byte = row_scale(amax, p.block);
                    const float sc = mx_inv_of_byte(byte);
                    const bool live = q_live && rl < rows;
                    if (live) {
                        uint32_t c[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) c[k] = codes4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], sc);
                        __stcs(reinterpret_cast<uint4*>(qp + 4 * j * p.ldq), make_uint4(c[0], c[1], c[2], c[3]));
                    }
                    if (!(lane & 1)) s_row[(rl & 31) * 16 + (rl >> 5) * 4 + ((lane & 7) >> 1)] = live ? static_cast<uint8_t>(byte) : 0;
                }
            }
        }
    }
    __syncthreads();
    if (p.q && threadIdx.x < 32) {
        const int64_t col_tiles = (cols32 + 127) / 128;
        reinterpret_cast<uint4*>(p.s + (rt * col_tiles + ct) * 512)[threadIdx.x] = reinterpret_cast<const uint4*>(s_row)[threadIdx.x];
    }
    if constexpr (SUM && !COL) {
        sum_columns<PACKED>(tile, sum_col);
        __syncthreads();
        store_sums(p, sum_col, c0, rt);
    }
    if constexpr (COL) {
        if constexpr (PACKED) {
            const int cp = threadIdx.x & 63, b = threadIdx.x >> 6;
            const int c = 2 * cp;
            uint32_t w[32];
            uint32_t m = 0u;
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = tile[(b * 32 + k) * (kQTile / 2) + cp];
            if constexpr (SUM) {
                float2 sum = both2(0.f);
#pragma unroll
                for (int k = 0; k < 32; ++k) sum = add2(sum, make_float2(lo_f32(w[k]), hi_f32(w[k])));
                sum_col[b][c] = sum.x;
                sum_col[b][c + 1] = sum.y;
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) m = max_abs2(m, w[k]);
            float a0 = fabsf(lo_f32(m)), a1 = fabsf(hi_f32(m));
            if (p.block == 128) {
                amax_col[b][c] = a0;
                amax_col[b][c + 1] = a1;
                __syncthreads();
                a0 = fmaxf(fmaxf(amax_col[0][c], amax_col[1][c]), fmaxf(amax_col[2][c], amax_col[3][c]));
                a1 = fmaxf(fmaxf(amax_col[0][c + 1], amax_col[1][c + 1]), fmaxf(amax_col[2][c + 1], amax_col[3][c + 1]));
            }
            const int y0 = mx_scale_byte(a0), y1 = mx_scale_byte(a1);
            const uint32_t sc = inv_of_byte_bf16(y0) | (inv_of_byte_bf16(y1) << 16);
            const bool row_live = r0 + b * 32 < rows32;
            const bool live0 = row_live && c0 + c < p.cols, live1 = row_live && c0 + c + 1 < p.cols;
            uint32_t x[8], y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t z[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) z[g] = mul2(w[4 * k + g], sc);
                x[k] = join(cvt_e4m3x2(lo_f32(z[0]), lo_f32(z[1])), cvt_e4m3x2(lo_f32(z[2]), lo_f32(z[3])));
                y[k] = join(cvt_e4m3x2(hi_f32(z[0]), hi_f32(z[1])), cvt_e4m3x2(hi_f32(z[2]), hi_f32(z[3])));
            }
            __syncthreads();  // the tile has been read
            stage_codes32(reinterpret_cast<uint4*>(tile), c, b, x);
            stage_codes32(reinterpret_cast<uint4*>(tile), c + 1, b, y);
            s_col[(c & 31) * 16 + (c >> 5) * 4 + b] = live0 ? static_cast<uint8_t>(y0) : 0;
            s_col[((c + 1) & 31) * 16 + (c >> 5) * 4 + b] = live1 ? static_cast<uint8_t>(y1) : 0;
        } else {
            const float* y = reinterpret_cast<const float*>(tile);
            constexpr int kBlocks = 4 * kQTile / kQThreads;  // 32-row blocks of its column per thread
            const int c = threadIdx.x & 127, b0 = (threadIdx.x >> 7) * kBlocks;
            const float* col = y + b0 * 32 * kQTile + 4 * swizzled(c >> 2) + (c & 3);
            float most = 0.f;
            if (p.block == 128) {
                float m = 0.f;
#pragma unroll 16
                for (int k = 0; k < 32 * kBlocks; ++k) m = fmaxf(m, fabsf(col[k * kQTile]));
                amax_col[threadIdx.x >> 7][c] = m;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 4 / kBlocks; ++k) most = fmaxf(most, amax_col[k][c]);
            }
            uint32_t x[kBlocks][8];
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                float w[32], amax = most;
#pragma unroll
                for (int k = 0; k < 32; ++k) w[k] = col[(j * 32 + k) * kQTile];
                if (p.block != 128) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) amax = fmaxf(amax, fabsf(w[k]));
                }
                if constexpr (SUM) {
                    float sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; ++k) sum += w[k];
                    sum_col[b0 + j][c] = sum;
                }
                const int byte = mx_scale_byte(amax);
                const float sc = mx_inv_of_byte(byte);
                s_col[(c & 31) * 16 + (c >> 5) * 4 + b0 + j] =
                    c0 + c < p.cols && r0 + (b0 + j) * 32 < rows32 ? static_cast<uint8_t>(byte) : 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) x[j][k] = codes4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3], sc);
            }
            __syncthreads();  // the tile has been read
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) stage_codes32(reinterpret_cast<uint4*>(tile), c, b0 + j, x[j]);
        }
        __syncthreads();
        if constexpr (SUM) store_sums(p, sum_col, c0, rt);
#pragma unroll
        for (int k = 0; k < kQTile; k += kQThreads / 8) {
            const int c = k + (threadIdx.x >> 3), piece = threadIdx.x & 7;
            if (c0 + c < p.cols && r0 + piece * 16 < rows32)
                __stcs(reinterpret_cast<uint4*>(p.qt + (c0 + c) * p.ldqt + r0) + piece,
                       reinterpret_cast<const uint4*>(tile)[c * 8 + (piece ^ stage_key(c))]);
        }
        if (threadIdx.x < 32) {
            const int64_t row_tiles = (rows32 + 127) / 128;
            reinterpret_cast<uint4*>(p.st + (ct * row_tiles + rt) * 512)[threadIdx.x] = reinterpret_cast<const uint4*>(s_col)[threadIdx.x];
        }
    }
}

// dbias from the row tiles' sums: 32 columns per CTA, G threads per column each adding
// every G-th tile in order, then the G in order.
template <int G>
__global__ void __launch_bounds__(32 * G) bias_sums_kernel(const float* sums, int tiles, int64_t cols, int accumulate, float* dbias) {
    __shared__ float red[G][33];
    wait_for_earlier_kernels();
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int k = g; k < tiles; k += G) s += sums[k * cols + col];
    red[g][c] = s;
    __syncthreads();
    if (g == 0 && col < cols) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < G; ++k) t += red[k][c];
        dbias[col] = accumulate ? dbias[col] + t : t;
    }
}

template <bool F32, bool PACKED, bool COL, bool SUM = false>
cudaError_t launch(const QuantArgs& a, cudaStream_t st) {
    constexpr int smem = !(COL || SUM) ? 0 : kQTile * kQTile * (PACKED ? 2 : 4);
    if (smem) {
        static PerDevice done;
        const cudaError_t e = allow_smem(quantize_kernel<F32, PACKED, COL, SUM>, smem, done);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>((a.rows + 127) / 128));
    note_launch();
    return launch_early(quantize_kernel<F32, PACKED, COL, SUM>, grid, kQThreads, smem, st, a);
}

}  // namespace

cudaError_t launch_bias_sums(const float* sums, int64_t tiles, int64_t cols, int accumulate, float* dbias, cudaStream_t st) {
    note_launch();
    const unsigned ctas = static_cast<unsigned>((cols + 31) / 32);
    // eight loads per thread: 64 tiles of 20480 columns in eight threads per column rather than 32
    const int n = static_cast<int>(tiles);
    if (n <= 64) return launch_early(bias_sums_kernel<8>, ctas, 256, 0, st, sums, n, cols, accumulate, dbias);
    return launch_early(bias_sums_kernel<32>, ctas, 1024, 0, st, sums, n, cols, accumulate, dbias);
}

cudaError_t launch_quantize(const QuantArgs& a, int f32, cudaStream_t st) {
    if (a.sums) {
        if (f32) return a.qt ? launch<true, false, true, true>(a, st) : launch<true, false, false, true>(a, st);
        return a.qt ? launch<false, true, true, true>(a, st) : launch<false, true, false, true>(a, st);
    }
    if (f32) return a.qt ? launch<true, false, true>(a, st) : launch<true, false, false>(a, st);
    if (a.row_mul || a.col_mul) return a.qt ? launch<false, false, true>(a, st) : launch<false, false, false>(a, st);
    return a.qt ? launch<false, true, true>(a, st) : launch<false, true, false>(a, st);
}

}  // namespace hm
