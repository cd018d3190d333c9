// Matrix product of MXFP8 operands on sm_103a tensor cores: D = A B^T with
// E4M3 codes and one UE8M0 scale per 1 x 32 block of each operand
//   D[m][n] = sum_b 2^(ea[m][b] + eb[n][b]) sum_{k in block b} A[m][k] B[n][k].
// tcgen05.mma kind::mxf8f6f4 applies the scales inside the tensor core: one
// MMA contracts K = 32, i.e. exactly one block of both operands, and reads
// the block's scales from TMEM, where tcgen05.cp puts them straight from the
// tiled scale layout (512 bytes hold the scales of 128 rows x 4 blocks: the
// image of 4 TMEM columns x 32 lanes, repeated for the four lane quadrants).
// Codes stream by TMA as 128-row x 128-byte tiles with the 128-byte swizzle,
// scales by 512-byte bulk copies onto the same mbarriers.
//
// Two kernels:
//   mx_gemm_kernel   persistent, 128 x 256 tiles of D, A's rows on the M side.
//   mx_gemm_split_kernel  few rows of A: B's rows take the M side (128 lanes),
//                    A's rows the N side (16 to 128 columns), and K is split
//                    over the CTAs of a cluster that add their parts through
//                    distributed shared memory in rank order.
// Every wait is bounded as in the Newton-Schulz kernels (HM_ERR_TIMEOUT in the
// device error word).
#include "hm.h"
#include "hm_internal.h"
#include "hm_ops.h"
#include "hm_ptx.cuh"

#include <cuda_bf16.h>

namespace hm {

namespace {

constexpr int kTileP = 128;      // rows of the M-side operand in a tile
constexpr int kTileK = 128;      // codes (bytes) of K per stage: four MMAs of K = 32
constexpr int kPBytes = kTileP * kTileK;
constexpr int kSfBytes = 512;    // scales of 128 rows x 4 blocks

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_cp_sf(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Shared-memory descriptor of one scale tile: 32 rows of 16 bytes, unswizzled,
// 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t desc_sf(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// kind::mxf8f6f4 instruction descriptor: E4M3 operands (0), K-major, UE8M0
// scales (bit 23), N >> 3 at bit 17, M >> 4 at bit 24.  The byte of the scale
// columns that an MMA uses is set at bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t mx_idesc(int m, int n) {
    return (1u << 23) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t sf_id(int kk) { return (static_cast<uint32_t>(kk) << 4) | (static_cast<uint32_t>(kk) << 29); }

__device__ __forceinline__ uint32_t bf16_pair(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------------------
// Epilogue of a 32-column chunk held one row per lane: D's row pointer plus
// the chunk's first column.  vec: bytes every row start is aligned to (32, 16
// or 0), so whole chunks leave as full 32-byte sectors.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store_chunk(const MxGemmArgs& p, int row, int col0, const uint32_t (&r)[32]) {
    if (row >= p.m || col0 >= p.n) return;
    const int64_t at = static_cast<int64_t>(row) * p.ldd + col0;
    const bool whole = col0 + 32 <= p.n;
    if (p.d_f32) {
        float* d = static_cast<float*>(p.d) + at;
        if (whole && p.vec >= 16) {
            float4* d4 = reinterpret_cast<float4*>(d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float4 v = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                       __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
                if (p.accumulate) {
                    const float4 o = d4[j];
                    v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                }
                d4[j] = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col0 + j < p.n) d[j] = p.accumulate ? d[j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
        }
    } else {
        uint16_t* d = static_cast<uint16_t*>(p.d) + at;
        if (whole && p.vec >= 16) {
            uint4* d4 = reinterpret_cast<uint4*>(d);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d4[j] = make_uint4(bf16_pair(r[8 * j], r[8 * j + 1]), bf16_pair(r[8 * j + 2], r[8 * j + 3]),
                                   bf16_pair(r[8 * j + 4], r[8 * j + 5]), bf16_pair(r[8 * j + 6], r[8 * j + 7]));
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (col0 + j < p.n) d[j] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[j])));
        }
    }
}

// ---------------------------------------------------------------------------
// Persistent kernel, 128 x 256 tiles, 320 threads:
//   warp 0      producer (one thread): codes by TMA, scales by bulk copies;
//   warp 1      owns TMEM, issues scale copies and MMAs (one thread);
//   warps 2-9   epilogue, two per TMEM lane quadrant, 128 columns each.
// TMEM (512 columns): two accumulators of 256 columns at 0 and 224, which
// share columns 224..255, and two slots of 12 scale columns at 480 and 496.
// The epilogue drains the shared columns of a tile first and then releases
// them, so the next tile's MMAs start while the rest is being stored.
// ---------------------------------------------------------------------------
constexpr int kBigN = 256;
constexpr int kBigStages = 4;
constexpr int kBigThreads = 320;
constexpr int kBigQBytes = kBigN * kTileK;
constexpr int kBigAcc1 = 224;
constexpr int kBigSf = 480;
constexpr int kBigSmem = kBigStages * (kPBytes + kBigQBytes + 3 * kSfBytes) + 1024 + 256;

__device__ __forceinline__ void big_tile(const MxGemmArgs& p, int t, int& tm, int& tn) {
    // bands of kGroup tile-rows, columns within a band: a band's A stays in L2
    constexpr int kGroup = 16;
    const int band = t / (kGroup * p.tiles_n);
    const int rows = min(kGroup, p.tiles_m - band * kGroup);
    const int l = t - band * kGroup * p.tiles_n;
    tm = band * kGroup + l % rows;
    tn = l / rows;
}

__global__ void __launch_bounds__(kBigThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                   const __grid_constant__ MxGemmArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sp = smem;
    uint8_t* sq = sp + kBigStages * kPBytes;
    uint8_t* ssf = sq + kBigStages * kBigQBytes;  // per stage: 512 bytes of A's scales, 1024 of B's
    uint64_t* full = reinterpret_cast<uint64_t*>(ssf + kBigStages * 3 * kSfBytes);
    uint64_t* empty = full + kBigStages;
    uint64_t* tfull = empty + kBigStages;  // two: accumulator written
    uint64_t* tfree = tfull + 2;           // shared columns of the current tile drained
    uint64_t* drain = tfree + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* bail = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kBigStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&tfull[0]), 1);
        mbar_init(smem_u32(&tfull[1]), 1);
        mbar_init(smem_u32(tfree), kBigThreads - 64);
        mbar_init(smem_u32(drain), 1);
        *bail = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = p.tiles_m * p.tiles_n;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                int tm, tn;
                big_tile(p, t, tm, tn);
                const int nsf = min(2, p.sf_rows_b - 2 * tn);  // B's scale tiles that exist
                const uint8_t* sfa = p.sa + static_cast<int64_t>(tm) * p.num_kb * kSfBytes;
                const uint8_t* sfb = p.sb + static_cast<int64_t>(2 * tn) * p.num_kb * kSfBytes;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, p.err, bail)) { ok = false; break; }
                    const uint32_t fb = smem_u32(&full[s]);
                    mbar_arrive_expect_tx(fb, kPBytes + kBigQBytes + kSfBytes * (1 + nsf));
                    tma_load_2d(smem_u32(sp + s * kPBytes), &tma, fb, kb * kTileK, tm * kTileP);
                    tma_load_2d(smem_u32(sq + s * kBigQBytes), &tmb, fb, kb * kTileK, tn * kBigN);
                    const uint32_t sf = smem_u32(ssf + s * 3 * kSfBytes);
                    bulk_load(sf, sfa + static_cast<int64_t>(kb) * kSfBytes, kSfBytes, fb);
                    for (int j = 0; j < nsf; ++j)
                        bulk_load(sf + kSfBytes * (1 + j), sfb + (static_cast<int64_t>(j) * p.num_kb + kb) * kSfBytes,
                                  kSfBytes, fb);
                    armed |= 1u << s;
                    armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    if (++s == kBigStages) { s = 0; ph ^= 1u; }
                }
            }
            // wait for this CTA's own copies still in flight
            for (int k = 0; k < kBigStages; ++k)
                if (armed & (1u << k)) mbar_wait(smem_u32(&full[k]), (armed_par >> k) & 1u, p.err, bail, false);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            int it = 0;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++it) {
                // tile it - 1 has released the shared columns (which also means
                // that tile it - 2, in this accumulator, was drained)
                if (it && !mbar_wait(smem_u32(tfree), (it - 1) & 1, p.err, bail)) break;
                tc_fence_after();
                const uint32_t d = tmem + ((it & 1) ? kBigAcc1 : 0);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&full[s]), ph, p.err, bail)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sf = smem_u32(ssf + s * 3 * kSfBytes);
                    const uint32_t tsf = tmem + kBigSf + slot * 16;
                    tmem_cp_sf(tsf, desc_sf(sf));
                    tmem_cp_sf(tsf + 4, desc_sf(sf + kSfBytes));
                    tmem_cp_sf(tsf + 8, desc_sf(sf + 2 * kSfBytes));
                    slot ^= 1;
                    const uint64_t ad = desc_sw128(smem_u32(sp + s * kPBytes));
                    const uint64_t bd = desc_sw128(smem_u32(sq + s * kBigQBytes));
                    // the last stage may hold fewer blocks: codes and scales past k are not used
                    const int nk = kb + 1 < p.num_kb ? 4 : p.last_nk;
                    for (int kk = 0; kk < nk; ++kk)
                        umma_mx(d, ad + 2 * kk, bd + 2 * kk, mx_idesc(kTileP, kBigN) | sf_id(kk), tsf, tsf + 4,
                                (kb | kk) != 0);
                    umma_commit(smem_u32(&empty[s]));
                    if (++s == kBigStages) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                umma_commit(smem_u32(&tfull[it & 1]));
            }
            // every MMA this thread issued has completed before TMEM is freed
            umma_commit(smem_u32(drain));
            mbar_wait(smem_u32(drain), 0, p.err, bail, false);
        }
    } else {
        const int q = warp & 3;            // TMEM lane quadrant of this warp
        const int half = (warp - 2) >> 2;  // which 128 of the tile's columns it drains
        int it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
            int tm, tn;
            big_tile(p, t, tm, tn);
            bool ok = mbar_wait(smem_u32(&tfull[it & 1]), (it >> 1) & 1, p.err, bail);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const int row = tm * kTileP + q * 32 + lane;
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + ((it & 1) ? kBigAcc1 : 0) + half * 128;
            // chunk order: accumulator 0 shares its last chunk, accumulator 1 its first
            const bool owner = half == ((it & 1) ? 0 : 1);
            if (!owner) {
                tc_fence_before();  // its loads of the previous tile
                mbar_arrive(smem_u32(tfree));
            }
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const int ch = (it & 1) ? c : 3 - c;
                uint32_t r[32];
                tmem_ld32(acc + ch * 32, r);
                tmem_ld_wait();
                tmem_ld_pin(r);
                if (c == 0 && owner) {
                    tc_fence_before();
                    mbar_arrive(smem_u32(tfree));
                }
                store_chunk(p, row, tn * kBigN + half * 128 + ch * 32, r);
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Split kernel: one tile of BN rows of A x 128 rows of B per cluster, K cut
// into one contiguous range of stages per CTA.  192 threads: producer warp, MMA
// warp, four epilogue warps.  B's rows are the M side, so a lane is a column
// of D and a warp's stores of one row of D are contiguous at any alignment.
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 192;

template <int BN>
struct SplitCfg {
    static constexpr int Q_BYTES = BN * kTileK;
    // two CTAs per SM: up to 113 KB each
    static constexpr int STAGES = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
    static constexpr int SMEM = STAGES * (kPBytes + Q_BYTES + 2 * kSfBytes) + 1024 + 256;
    static constexpr int ACC = BN < 32 ? 32 : BN;
    static constexpr int TMEM = ACC <= 32 ? 64 : 2 * ACC;  // accumulator and two slots of 8 scale columns
    static_assert(STAGES * (kPBytes + Q_BYTES) >= BN * 128 * 4, "the ring holds the partial tile");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store_one(const MxGemmArgs& p, int row, int col, float v) {
    const int64_t at = static_cast<int64_t>(row) * p.ldd + col;
    if (p.d_f32) {
        float* d = static_cast<float*>(p.d) + at;
        *d = p.accumulate ? *d + v : v;
    } else {
        static_cast<uint16_t*>(p.d)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

template <int BN>
__global__ void __launch_bounds__(kSplitThreads)
    mx_gemm_split_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                         const __grid_constant__ MxGemmArgs p) {
    using C = SplitCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sp = smem;                            // B's rows
    uint8_t* sq = sp + C::STAGES * kPBytes;        // A's rows
    uint8_t* ssf = sq + C::STAGES * C::Q_BYTES;    // per stage: 512 bytes of B's scales, 512 of A's
    uint64_t* full = reinterpret_cast<uint64_t*>(ssf + C::STAGES * 2 * kSfBytes);
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
    volatile int* bail = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* part = reinterpret_cast<float*>(smem);  // [BN][128], over the ring once it has been read

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int ck = p.split, rank = ck > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tp = blockIdx.x / ck, tq = blockIdx.y;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / ck);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / ck);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        *bail = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            const uint8_t* sfp = p.sb + static_cast<int64_t>(tp) * p.num_kb * kSfBytes;
            const uint8_t* sfq = p.sa + static_cast<int64_t>(tq * BN / 128) * p.num_kb * kSfBytes;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, p.err, bail)) break;
                const uint32_t fb = smem_u32(&full[s]);
                mbar_arrive_expect_tx(fb, kPBytes + C::Q_BYTES + 2 * kSfBytes);
                tma_load_2d(smem_u32(sp + s * kPBytes), &tmb, fb, kb * kTileK, tp * kTileP);
                tma_load_2d(smem_u32(sq + s * C::Q_BYTES), &tma, fb, kb * kTileK, tq * BN);
                const uint32_t sf = smem_u32(ssf + s * 2 * kSfBytes);
                bulk_load(sf, sfp + static_cast<int64_t>(kb) * kSfBytes, kSfBytes, fb);
                bulk_load(sf + kSfBytes, sfq + static_cast<int64_t>(kb) * kSfBytes, kSfBytes, fb);
                armed |= 1u << s;
                armed_par = (armed_par & ~(1u << s)) | (ph << s);
                if (++s == C::STAGES) { s = 0; ph ^= 1u; }
            }
            for (int k = 0; k < C::STAGES; ++k)
                if (armed & (1u << k)) mbar_wait(smem_u32(&full[k]), (armed_par >> k) & 1u, p.err, bail, false);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, slot = 0;
            uint32_t ph = 0;
            const uint32_t sfq_col = static_cast<uint32_t>(tq * BN % 128) / 32;  // A's rows inside its 128-row scale tile
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(smem_u32(&full[s]), ph, p.err, bail)) break;
                tc_fence_after();
                const uint32_t sf = smem_u32(ssf + s * 2 * kSfBytes);
                const uint32_t tsf = tmem + C::ACC + slot * 8;
                tmem_cp_sf(tsf, desc_sf(sf));
                tmem_cp_sf(tsf + 4, desc_sf(sf + kSfBytes));
                slot ^= 1;
                const uint64_t pd = desc_sw128(smem_u32(sp + s * kPBytes));
                const uint64_t qd = desc_sw128(smem_u32(sq + s * C::Q_BYTES));
                const int nk = kb + 1 < p.num_kb ? 4 : p.last_nk;
                for (int kk = 0; kk < nk; ++kk)
                    umma_mx(tmem, pd + 2 * kk, qd + 2 * kk, mx_idesc(kTileP, BN) | sf_id(kk), tsf, tsf + 4 + sfq_col,
                            (kb - kb0) | kk);
                umma_commit(smem_u32(&empty[s]));
                if (++s == C::STAGES) { s = 0; ph ^= 1u; }
            }
            // also covers every MMA issued before an early exit
            umma_commit(smem_u32(tfull));
            mbar_wait(smem_u32(tfull), 0, p.err, bail, false);
        }
    }
    __syncwarp();
    // the epilogue warps wait for the accumulator; the others only join the barriers below
    const int q = warp & 3;
    const int col = tp * kTileP + q * 32 + lane;  // column of D
    const int row0 = tq * BN;
    const int rows = min(BN, p.m - row0);
    if (warp >= 2) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(tfull), 0, p.err, bail));
        tc_fence_after();
        if (ok) {
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, r);
                tmem_ld_wait();
                tmem_ld_pin(r);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j >= rows) break;
                    if (ck > 1) part[(c0 + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
                    else if (col < p.n) store_one(p, row0 + c0 + j, col, __uint_as_float(r[j]));
                }
            }
        }
        tc_fence_before();
    }
    if (ck > 1) {
        cluster_sync_all();
        // rows of D dealt round-robin over the cluster; every part in rank order
        if (warp >= 2 && col < p.n) {
            const uint32_t mine = smem_u32(part) + static_cast<uint32_t>(q * 32 + lane) * 4;
            for (int c = rank; c < rows; c += ck) {
                float v = 0.f;
                for (int k = 0; k < ck; ++k) v += ld_cluster_f32(mapa_shared(mine + c * 512, k));
                store_one(p, row0 + c, col, v);
            }
        }
        cluster_sync_all();  // a CTA's part stays until its peers have read it
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// K = 0: the sum is empty.
__global__ void __launch_bounds__(256) mx_gemm_zero_kernel(const __grid_constant__ MxGemmArgs p) {
    const int64_t total = static_cast<int64_t>(p.m) * p.n;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll)
        store_one(p, static_cast<int>(i / p.n), static_cast<int>(i % p.n), 0.f);
}

// Codes [rows][ld], k of them used: boxes of box_rows x 128 bytes, zero outside.
bool map_codes(CUtensorMap* m, const uint8_t* base, int64_t k, int64_t rows, int64_t ld, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {kTileK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, bool (&done)[64]) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    return cudaSuccess;
}

template <int BN>
cudaError_t launch_split(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, MxGemmArgs p, cudaStream_t st) {
    using C = SplitCfg<BN>;
    static bool done[64] = {false};
    cudaError_t e = allow_smem(mx_gemm_split_kernel<BN>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mb;
    if (!map_codes(&ma, a, p.k, p.m, lda, BN) || !map_codes(&mb, b, p.k, p.n, ldb, kTileP)) return cudaErrorUnknown;
    const int tiles_p = (p.n + kTileP - 1) / kTileP, tiles_q = (p.m + BN - 1) / BN;
    // enough CTAs for two per SM, at least two stages each
    int split = 1;
    while (split < 8 && 2 * split * tiles_p * tiles_q <= 2 * device_sm_count() && 4 * split <= p.num_kb) split *= 2;
    p.split = split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles_p * split, tiles_q, 1);
    cfg.blockDim = dim3(kSplitThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    note_launch();
    return cudaLaunchKernelEx(&cfg, mx_gemm_split_kernel<BN>, ma, mb, p);
}

}  // namespace

cudaError_t launch_mx_gemm(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, const MxGemmArgs& args,
                           cudaStream_t st) {
    MxGemmArgs p = args;
    if (p.k == 0) {
        if (p.accumulate) return cudaSuccess;
        const int64_t blocks = (static_cast<int64_t>(p.m) * p.n + 255) / 256;
        note_launch();
        mx_gemm_zero_kernel<<<resident_grid(mx_gemm_zero_kernel, 256, blocks), 256, 0, st>>>(p);
        return cudaGetLastError();
    }
    p.num_kb = (p.k + kTileK - 1) / kTileK;
    p.last_nk = (p.k - (p.num_kb - 1) * kTileK) / 32;
    p.sf_rows_b = (p.n + 127) / 128;
    p.err = device_error_word();
    const int64_t row_bytes = p.ldd * (p.d_f32 ? 4 : 2);
    p.vec = (reinterpret_cast<uintptr_t>(p.d) | static_cast<uintptr_t>(row_bytes)) % 16 == 0 ? 16 : 0;
    if (p.m <= 16) return launch_split<16>(a, lda, b, ldb, p, st);
    if (p.m <= 32) return launch_split<32>(a, lda, b, ldb, p, st);
    if (p.m <= 64) return launch_split<64>(a, lda, b, ldb, p, st);
    if (p.m <= 128) return launch_split<128>(a, lda, b, ldb, p, st);
    static bool done[64] = {false};
    cudaError_t e = allow_smem(mx_gemm_kernel, kBigSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mb;
    if (!map_codes(&ma, a, p.k, p.m, lda, kTileP) || !map_codes(&mb, b, p.k, p.n, ldb, kBigN)) return cudaErrorUnknown;
    p.tiles_m = (p.m + kTileP - 1) / kTileP;
    p.tiles_n = (p.n + kBigN - 1) / kBigN;
    const int64_t total = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    const int grid = static_cast<int>(total < device_sm_count() ? total : device_sm_count());
    note_launch();
    mx_gemm_kernel<<<grid, kBigThreads, kBigSmem, st>>>(ma, mb, p);
    return cudaGetLastError();
}

}  // namespace hm
