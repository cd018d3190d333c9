// Internal declarations of the operators around the update (MXFP8 product,
// quantization, RMS norm, gradient clipping): kernel arguments and launchers.
// Not part of the C ABI.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace hm {

// Lets a kernel use `bytes` of dynamic shared memory, once per device.
using PerDevice = std::atomic<bool>[64];
template <class Kernel>
inline cudaError_t allow_smem(Kernel kernel, int bytes, PerDevice& done) {
    int dev = 0;
    cudaGetDevice(&dev);
    const bool keep = dev >= 0 && dev < 64;
    if (keep && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && keep) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

// A launch that may be set up while the kernel before it drains; the kernel calls
// wait_for_earlier_kernels() before it touches global memory, and reads it with
// ordinary loads: the read-only path (__ldg, const __restrict__) is for data that
// nobody writes while the kernel runs.  One call after
// another: RMS norm 8192 x 5120 49.0 -> 46.0 us, its gradient (two kernels) 59.9 ->
// 54.8, quantization 8192 x 15360 81.9 -> 79.6, clipping of 200,000 elements 10.2 ->
// 8.2.
template <class... Params, class... Args>
inline cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct MxGemmArgs {
    const uint8_t* sa;   // tiled scales
    const uint8_t* sb;
    void* d;
    int64_t ldd;         // elements
    int32_t m, n, k;
    int32_t d_f32, accumulate;
    // filled in by launch_mx_gemm
    int32_t num_kb;      // stages of 128 along K
    int32_t last_nk;     // blocks of 32 in the last stage
    int32_t tiles_p, tiles_q;  // pair kernel: tiles along n and m
    int32_t split;       // split kernel: CTAs of a cluster that share K
    int32_t inject;      // failure test: never signal an accumulator as ready
    int32_t* err;
};
// Which kernel a product takes: `tile` rows of A per tile, K over `parts` CTAs of a
// cluster (0: the pair kernel), there with `sums` of chunks of K in registers.
struct MxGemmForm {
    int32_t tile, parts, sums;
};
cudaError_t mx_gemm_form(const MxGemmArgs& p, MxGemmForm* f);  // m, n, k, d_f32 of p, k > 0
// Failure-detection test hook: HM_INJECT_MX_WAIT_TIMEOUT=1 in the environment makes
// the waits of the product and of the norm's gradient run out (bounded), so that
// they record HM_ERR_TIMEOUT.
bool inject_mx_timeout();
cudaError_t launch_mx_gemm(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, const MxGemmArgs& args,
                           cudaStream_t st);

struct QuantArgs {
    const void* x;
    int64_t rows, cols, ldx;
    const float* row_mul;
    const float* col_mul;
    uint8_t* q;          // [rows][ldq] or nullptr
    int64_t ldq;
    uint8_t* s;
    uint8_t* qt;         // [cols][ldqt] or nullptr
    int64_t ldqt;
    uint8_t* st;
    int32_t block;       // 32 or 128
    int32_t vec;         // x's rows are 16-byte aligned
    int32_t col_vec;     // there are column factors, 16-byte aligned
    int32_t pad;
};
cudaError_t launch_quantize(const QuantArgs& a, int f32, cudaStream_t st);

struct RmsArgs {
    const void* x;       // [rows][ldx]
    const void* res;     // [rows][ldh] or nullptr
    void* h;             // [rows][ldh] or nullptr
    int64_t ldx, ldh, rows;
    int32_t d, block;
    const float* gamma;
    float eps;
    float* rstd;
    uint8_t* q;          // [rows][d]
    uint8_t* s;
};
cudaError_t launch_rmsnorm(const RmsArgs& a, int f32, cudaStream_t st);

struct RmsGradArgs {
    const void* dy;      // [rows][lddy]
    const void* dres;    // [rows][ldh] or nullptr
    const void* h;
    void* dx;
    int64_t lddy, ldh, rows;
    int32_t d, accumulate;
    const float* gamma;
    const float* rstd;
    float* dgamma;
    float* partials;     // [CTAs][d]
    int32_t stages;      // rows in flight per CTA (set by launch_rmsnorm_grad, as err)
    int32_t inject;      // failure test: never load a row
    int32_t* err;
};
// CTAs (= partial rows of dgamma) that launch_rmsnorm_grad uses, at most
int rmsnorm_grad_parts(int64_t rows, int64_t d);
cudaError_t launch_rmsnorm_grad(const RmsGradArgs& a, int f32, cudaStream_t st);

// A launch takes its tensors by value: up to kClipTensors, or up to kClipFew in
// the one-launch form for little data.
constexpr int kClipTensors = 256;
constexpr int kClipFew = 16;
struct ClipTensor {
    const void* src;
    void* dst;           // nullptr: only counted
    int64_t n;
    int32_t first;       // chunks before this tensor
    int32_t f32;
};
struct ClipHead {
    int32_t n;           // tensors
    int32_t chunks;
    int32_t parts;       // partial sums of every launch of the call together
    int32_t part0;       // this launch's first one
    int32_t keep_from;   // norm pass: chunks from here on stay in the L2 (set by launch_clip_norm)
    int32_t pad;
    float max_norm, eps;
    float* stats;
    double* partials;
};
template <int CAP>
struct ClipArgs {
    ClipHead h;
    ClipTensor t[CAP];
};
constexpr int kClipChunkVecs = 4096;       // 16-byte vectors per chunk
constexpr int kClipFewChunkVecs = 1024;    // in the one-launch form,
constexpr int kClipFewChunks = 64;         // which takes at most so many (1 MB)
int clip_chunks(const void* src, int64_t n, int f32, int vecs);  // of one tensor with n > 0
int clip_parts(int chunks);                                      // partial sums of one launch
cudaError_t launch_clip_norm(ClipArgs<kClipTensors>& a, cudaStream_t st);
cudaError_t launch_clip_scale(const ClipArgs<kClipTensors>& a, cudaStream_t st);
cudaError_t launch_clip_few(const ClipArgs<kClipFew>& a, cudaStream_t st);

}  // namespace hm
