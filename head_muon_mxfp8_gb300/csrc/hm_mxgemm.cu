// Matrix product of MXFP8 operands on sm_103a tensor cores: D = A B^T with
// E4M3 codes and one UE8M0 scale per 1 x 32 block of each operand
//   D[m][n] = sum_b 2^(ea[m][b] + eb[n][b]) sum_{k in block b} A[m][k] B[n][k].
// tcgen05.mma kind::mxf8f6f4 applies the scales inside the tensor core: one
// MMA contracts K = 32, i.e. exactly one block of both operands, and reads
// the block's scales from TMEM, where tcgen05.cp puts them straight from the
// tiled scale layout (512 bytes hold the scales of 128 rows x 4 blocks: the
// image of 4 TMEM columns x 32 lanes, repeated for the four lane quadrants).
// Codes stream by TMA as 128-row x 128-byte tiles with the 128-byte swizzle,
// scales as 512-byte images onto the same mbarriers (TMA boxes in the pair
// kernel, bulk copies in the split kernel).
//
// Two kernels:
//   mx_gemm_pair_kernel   persistent CTA pairs, tiles of 256 x 128 to 256.
//   mx_gemm_split_kernel  few rows of A: B's rows take the M side (128 lanes),
//                    A's rows the N side (16 to 128 columns), and K is split
//                    over the CTAs of a cluster (2 to 8) that add their parts through
//                    distributed shared memory in rank order.
// Bound by: large products by the power cap, so their time goes with the clock that the
// operands' bits leave (8192 x 20480 x 5120 to bf16, codes of random bits: 580 us, 2.96 PFLOP/s at
// 1372 MHz median); 6144 x 4096 x 4096 added to fp32, 92 us, by the
// loads into the SMs and by D; a token's row by latency (1 x 5120 x 5120: 6.4 us,
// 4.0 at the copy rate).
// With an epilogue (hm_epilogue.cuh), calls of all kinds in turn on those operands and at that
// clock: plain 580 us, without activation 618, with bias, GELU and the kept sum 657, as its
// gradient 681, both of a gated pair's 713.
// Every wait is bounded as in the Newton-Schulz kernels (HM_ERR_TIMEOUT in the
// device error word).
#include "hm.h"
#include "hm_epilogue.cuh"
#include "hm_internal.h"
#include "hm_ops.h"
#include "hm_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

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
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int c0,
                                                 int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_cp_sf_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------------------
// Epilogue of a 32-column chunk of a tile: lane = column i of D, register j =
// row j0 + j.  A warp's lanes store neighbours in one row of D: one line per
// instruction at any alignment and pitch.  With A's rows on the M side instead
// (a lane holding 32 columns of its row, stored as 32-byte sectors) an
// instruction touched 32 lines: adding a 256 x 192 fp32 tile to D took 16,000
// clocks instead of the 4,100 of a 1024-long chunk of its products.
// ---------------------------------------------------------------------------
template <bool TAIL>
__device__ __forceinline__ void store_rows(const MxGemmArgs& p, int i, int j0, const uint32_t (&r)[32]) {
    const int rows = p.m - j0;  // TAIL: fewer than 32
    const int64_t at = static_cast<int64_t>(j0) * p.ldd + i;
    if (!p.d_f32) {
        uint16_t* d = static_cast<uint16_t*>(p.d) + at;
#pragma unroll
        for (int j = 0; j < 32; ++j, d += p.ldd)
            if (!TAIL || j < rows) *d = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(r[j])));
        return;
    }
    float* d = static_cast<float*>(p.d) + at;
    constexpr int kBatch = TAIL ? 8 : 32;  // a batch's loads before its first store (the tail's short ones save registers)
#pragma unroll
    for (int b = 0; b < 32; b += kBatch) {
        float old[kBatch];
        if (p.accumulate) {
            const float* o = d;
#pragma unroll
            for (int j = 0; j < kBatch; ++j, o += p.ldd) old[j] = !TAIL || b + j < rows ? *o : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j, d += p.ldd)
            if (!TAIL || b + j < rows) *d = p.accumulate ? old[j] + __uint_as_float(r[b + j]) : __uint_as_float(r[b + j]);
    }
}

__device__ __forceinline__ void store_chunk(const MxGemmArgs& p, int i, int j0, const uint32_t (&r)[32]) {
    if (i >= p.n || j0 >= p.m) return;
    if (j0 + 32 <= p.m) store_rows<false>(p, i, j0, r);
    else store_rows<true>(p, i, j0, r);
}

// ---------------------------------------------------------------------------
// Persistent kernel on CTA pairs (cta_group::2), tiles of 256 M-side rows (B's
// rows, D's columns) x BN N-side rows (A's, D's rows), 320 threads per CTA.  Each CTA of a pair loads its 128 M-side rows
// and half of the N-side rows; the even one issues the MMAs, which read both
// CTAs' shared memory and leave 128 rows x BN columns in each CTA's TMEM.  The
// scales of all BN N-side rows are needed by both CTAs, those of the M-side rows
// by their own.
//   warp 0      producer (one thread): codes and scales by TMA, both CTAs'
//               copies counted on the even CTA's barrier;
//   warp 1      owns TMEM; in the even CTA issues scale copies and MMAs;
//   warps 2-9   epilogue, two per TMEM lane quadrant, every other 32 columns.
// TMEM (512 columns): two accumulators and, from column 480, two slots of 16
// scale columns.  For BN = 256 the accumulators (at 0 and 224) share columns
// 224..255: the epilogue drains those first and releases them, and the next
// tile's MMAs start then.  For BN <= 192 they are disjoint.
//
// SUMS (fp32 D, K > kChunkK): the tensor core truncates when it adds a product
// to an accumulator, a bias towards zero that grows with the number of additions
// (relative error of a 6144 x 4096 weight gradient over 4096 tokens: 1.7e-6 with
// one sum over all of K, 2.0e-7 in chunks of 2048, 1.1e-7 in chunks of 1024; a
// plain fp32 product 2.5e-7; on another input 1.3e-7 in chunks of 2048 and 0.8e-7 plain).  A tile's K is then cut into chunks of 2048,
// accumulated alternately in the two accumulators, and the epilogue adds the
// chunks in registers with rounding to nearest while the next one runs.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 320;
constexpr int kPairEpiWarps = kPairThreads / 32 - 2;
constexpr int kChunkK = 2048;
constexpr int kSfCol = 480;

template <int BN>
struct PairMx {
    static constexpr int STAGES = BN == 256 ? 6 : BN == 128 ? 8 : 7;
    static constexpr int Q_BYTES = BN / 2 * kTileK;               // this CTA's half of the N side
    static constexpr int NSF = (BN + 127) / 128;                  // 128-row scale tiles that BN rows from a multiple of 64 touch
    static constexpr int SF_BYTES = (1 + NSF) * kSfBytes;
    static constexpr int STAGE_BYTES = kPBytes + Q_BYTES + SF_BYTES;
    static constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + 256;
    static constexpr int ACC1 = BN == 256 ? 224 : BN;
    static constexpr int CHUNKS = BN / 32;
    // scale columns are addressed at even offsets only: BN a multiple of 64
    static_assert(BN % 64 == 0 && SMEM <= 232448 && ACC1 + BN <= kSfCol, "pair tile");
};

__device__ __forceinline__ void pair_tile(const MxGemmArgs& p, int t, int& tp, int& tq) {
    // bands of 8 256-row M-side tiles, N-side tiles within a band
    constexpr int kGroup = 8;
    const int band = t / (kGroup * p.tiles_q);
    const int rows = min(kGroup, p.tiles_p - band * kGroup);
    const int l = t - band * kGroup * p.tiles_q;
    tp = band * kGroup + l % rows;
    tq = l / rows;
}

template <int BN, bool SUMS, int EPI>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap mp, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap msp, const __grid_constant__ CUtensorMap msq,
                        const __grid_constant__ MxGemmArgs p) {
    using C = PairMx<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sp = smem;
    uint8_t* sq = sp + C::STAGES * kPBytes;
    uint8_t* ssf = sq + C::STAGES * C::Q_BYTES;  // per stage: the M side's scale tile, then the N side's NSF
    uint64_t* full = reinterpret_cast<uint64_t*>(ssf + C::STAGES * C::SF_BYTES);
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tfree = tfull + 2;
    uint64_t* drain = tfree + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* bail = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank() & 1u;
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&tfull[b]), 1);
            mbar_init(smem_u32(&tfree[b]), 2 * kPairEpiWarps);
        }
        mbar_init(smem_u32(drain), 1);
        *bail = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    __syncwarp();  // thread 0's set-up is behind its warp: the barrier is taken by whole warps
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    wait_for_earlier_kernels();
    const uint32_t tmem = *tmem_slot;
    const int total = p.tiles_p * p.tiles_q;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    // a unit: the part of a tile's K that one accumulator sums
    const int unit_kb = SUMS ? kChunkK / kTileK : p.num_kb;
    const int units = SUMS ? (p.num_kb + unit_kb - 1) / unit_kb : 1;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, armed = 0, armed_par = 0;
            bool ok = true;
            for (int t = pair; t < total && ok; t += npairs) {
                int tp, tq;
                pair_tile(p, t, tp, tq);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, p.err, bail)) { ok = false; break; }
                    armed |= 1u << s;
                    armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
                    if (leader) mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * C::STAGE_BYTES);
                    tma_load_2d_pair(smem_u32(sp + s * kPBytes), &mp, fb, kb * kTileK, tp * 256 + rank * 128);
                    tma_load_2d_pair(smem_u32(sq + s * C::Q_BYTES), &mq, fb, kb * kTileK, tq * BN + rank * (BN / 2));
                    const uint32_t sf = smem_u32(ssf + s * C::SF_BYTES);
                    tma_load_3d_pair(sf, &msp, fb, 0, kb, tp * 2 + rank);
                    tma_load_3d_pair(sf + kSfBytes, &msq, fb, 0, kb, tq * BN / 128);
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            // the even CTA's full barriers count both CTAs' bytes: waiting on
            // them covers every copy of the pair still in flight
            if (leader)
                for (int k = 0; k < C::STAGES; ++k)
                    if (armed & (1u << k)) mbar_wait(smem_u32(&full[k]), (armed_par >> k) & 1u, p.err, bail, false);
        }
    } else if (warp == 1) {
        if (leader) {
            // the whole warp walks the loop (its waits and descriptors are warp-uniform)
            // and one elected lane issues: with a single lane in the loop the issue of a
            // stage's copies and MMAs took longer than the MMAs themselves
            int s = 0, slot = 0, u = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint64_t pd0 = desc_sw128(smem_u32(sp)), qd0 = desc_sw128(smem_u32(sq)), sd0 = desc_sf(smem_u32(ssf));
            for (int t = pair; t < total && ok; t += npairs) {
                int tp, tq;
                pair_tile(p, t, tp, tq);
                const uint32_t sfq_col = static_cast<uint32_t>(tq * BN % 128) / 32;  // the tile's rows inside its scale tiles
                for (int c = 0; c < units && ok; ++c, ++u) {
                    // BN = 256: unit u - 1 has released the shared columns, so unit u - 2
                    // (this accumulator's last) is drained too; else unit u - 2 is drained
                    if (BN == 256) {
                        if (u >= 1) ok = mbar_wait(smem_u32(&tfree[(u - 1) & 1]), ((u - 1) >> 1) & 1, p.err, bail);
                    } else {
                        if (u >= 2) ok = mbar_wait(smem_u32(&tfree[u & 1]), ((u >> 1) - 1) & 1, p.err, bail);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + ((u & 1) ? C::ACC1 : 0);
                    const int kb0 = c * unit_kb, kb1 = min(kb0 + unit_kb, p.num_kb);
                    for (int kb = kb0; kb < kb1; ++kb) {
                        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), ph, p.err, bail));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t tsf = tmem + kSfCol + slot * 16;
                        const uint64_t pd = pd0 + static_cast<uint64_t>(s * (kPBytes >> 4));
                        const uint64_t qd = qd0 + static_cast<uint64_t>(s * (C::Q_BYTES >> 4));
                        const uint64_t sd = sd0 + static_cast<uint64_t>(s * (C::SF_BYTES >> 4));
                        // the last stage may hold fewer blocks: codes and scales past k are not used
                        const int nk = kb + 1 < p.num_kb ? 4 : p.last_nk;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k <= C::NSF; ++k) tmem_cp_sf_pair(tsf + 4 * k, sd + k * (kSfBytes >> 4));
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                if (kk < nk)
                                    umma_mx_pair(d, pd + 2 * kk, qd + 2 * kk, mx_idesc(256, BN) | sf_id(kk), tsf,
                                                 tsf + 4 + sfq_col, (kb - kb0) | kk);
                            umma_commit_pair(smem_u32(&empty[s]));
                            if (kb + 1 == kb1 && !p.inject) umma_commit_pair(smem_u32(&tfull[u & 1]));
                        }
                        __syncwarp();
                        slot ^= 1;
                        if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                    }
                }
            }
            // every MMA this warp issued has completed before TMEM is freed
            if (elect_one()) {
                umma_commit_pair(smem_u32(drain));
                mbar_wait(smem_u32(drain), 0, p.err, bail, false);
            }
            __syncwarp();
        }
    } else {
        const int q = warp & 3;            // TMEM lane quadrant of this warp
        const int half = (warp - 2) >> 2;  // takes the chunks of this parity
        // one relaxed arrival per warp: it hands back TMEM columns that were read, no
        // memory, and a release at cluster scope held each one for 2,000 clocks
        auto release = [&](uint32_t bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(bar);
        };
        const uint32_t free0 = mapa_shared(smem_u32(&tfree[0]), 0), free1 = mapa_shared(smem_u32(&tfree[1]), 0);
        // with an epilogue: this warp's place for turning pieces, its pieces of a tile and
        // where the k-th begins (the owner of BN = 256's shared columns starts with those)
        float* stage = reinterpret_cast<float*>(smem_raw + C::SMEM) + (warp - 2) * (kPieceBytes / 4);
        constexpr int kPieces = (C::CHUNKS + 1) / 2 * 2;
        auto piece_at = [&](int k, int unit) {
            const int order = BN == 256 && !(unit & 1) ? (C::CHUNKS + 1) / 2 - 1 - (k >> 1) : k >> 1;
            return (2 * order + half) * 32 + (k & 1) * 16;
        };
        int u = 0;
        bool ok = true;
        for (int t = pair; t < total && ok; t += npairs) {
            int tp, tq;
            pair_tile(p, t, tp, tq);
            const int i = tp * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
            float sum[SUMS ? (C::CHUNKS + 1) / 2 : 1][32];
            EpiPiece<EPI, !SUMS, SUMS> piece;
            float2 bias[4];
            if constexpr (EPI != kEpiNone) {
                piece.bias(p, i - lane, bias);
                if (!SUMS) piece.load(p, tq * BN + piece_at(0, u), i - lane);
            }
            if (EPI) {
                // what the epilogue reads, likewise (see below)
#pragma unroll
                for (int ch = half; ch < C::CHUNKS; ch += 2) {
                    const int64_t row = tq * BN + ch * 32 + lane;
                    if (i - lane >= p.n || row >= p.m) continue;
                    const int es = p.d_f32 ? 4 : 2;
                    if (p.e.in) prefetch_l2(static_cast<const char*>(p.e.in) + (row * p.e.ld_in + (i - lane)) * es);
                    if (p.e.in2) prefetch_l2(static_cast<const char*>(p.e.in2) + (row * p.e.ld_in2 + (i - lane)) * es);
                }
            } else if (p.accumulate) {
                // the earlier D is read when the tile is done: start it into the L2
                // now, lane l the line of row l of each chunk
#pragma unroll
                for (int ch = half; ch < C::CHUNKS; ch += 2)
                    if (i - lane < p.n && tq * BN + ch * 32 + lane < p.m)
                        prefetch_l2(static_cast<const float*>(p.d) +
                                    static_cast<int64_t>(tq * BN + ch * 32 + lane) * p.ldd + (i - lane));
            }
            for (int c = 0; c < units; ++c, ++u) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[u & 1]), (u >> 1) & 1, p.err, bail));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + ((u & 1) ? C::ACC1 : 0);
                const uint32_t freed = (u & 1) ? free1 : free0;
                // BN = 256: accumulator 0 shares its last chunk (odd half), accumulator 1 its
                // first (even half); that half drains it first, the other has nothing to release
                const bool owner = BN == 256 && half == ((u & 1) ? 0 : 1);
                if (BN == 256 && !owner) release(freed);
                if constexpr (EPI && !SUMS) {
                    // one copy of the epilogue's code: a piece of 16 columns of the accumulator at a time
#pragma unroll 1
                    for (int k = 0; k < kPieces; ++k) {
                        const int at = piece_at(k, u), next = piece_at(k + 1, u);
                        if (at >= BN) break;
                        piece.begin(p, tq * BN + at, i - lane);
                        uint32_t r[16];
                        __syncwarp();
                        tmem_ld16(acc + at, r);
                        tmem_ld_wait();
                        tmem_ld_pin16(r);
                        if (owner && k == 1) release(freed);
                        EpiPiece<EPI, true, false> ahead;
                        if (k + 1 < kPieces && next < BN) ahead.load(p, tq * BN + next, i - lane);
                        piece.finish(p, stage, tq * BN + at, i - lane, bias, r);
                        piece.take(p, ahead);
                    }
                    if (BN != 256) release(freed);
                } else {
#pragma unroll
                    for (int k = 0; k < (C::CHUNKS + 1) / 2; ++k) {
                        const int order = BN == 256 && !(u & 1) ? (C::CHUNKS + 1) / 2 - 1 - k : k;
                        const int ch = 2 * order + half;
                        if (ch >= C::CHUNKS) break;
                        if (SUMS) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t r[16];
                                __syncwarp();
                                tmem_ld16(acc + ch * 32 + h * 16, r);
                                tmem_ld_wait();
                                tmem_ld_pin16(r);
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float v = __uint_as_float(r[j]);
                                    sum[k][16 * h + j] = c ? sum[k][16 * h + j] + v : v;
                                }
                            }
                            continue;
                        }
                        uint32_t r[32];
                        __syncwarp();  // lanes past the last column left the chunk before early
                        tmem_ld32(acc + ch * 32, r);
                        tmem_ld_wait();
                        tmem_ld_pin(r);
                        if (owner && k == 0) release(freed);
                        store_chunk(p, i, tq * BN + ch * 32, r);
                    }
                    if (BN != 256) release(freed);
                }
            }
            if (SUMS && EPI != kEpiNone && ok) {
#pragma unroll 1
                for (int k = 0; k < kPieces; ++k) {
                    const int at = (2 * (k >> 1) + half) * 32 + (k & 1) * 16;
                    if (at >= BN) break;
                    uint32_t r[16];
#pragma unroll
                    for (int c = 0; c < kPieces; ++c)
                        if (c == k)
#pragma unroll
                            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(sum[(c >> 1) % (SUMS ? kPieces / 2 : 1)][16 * (c & 1) + j]);
                    piece.begin(p, tq * BN + at, i - lane);
                    piece.finish(p, stage, tq * BN + at, i - lane, bias, r);
                }
            } else if (SUMS && ok) {
#pragma unroll
                for (int k = 0; k < (C::CHUNKS + 1) / 2; ++k) {
                    const int ch = 2 * k + half;
                    if (ch >= C::CHUNKS) break;
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(sum[k][j]);
                    store_chunk(p, i, tq * BN + ch * 32, r);
                }
            }
        }
    }
    // the peer's MMAs read this CTA's shared memory and write its TMEM: keep
    // both alive until every role of both CTAs is done
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Split kernel: one tile of BN rows of A x 128 rows of B per cluster, K cut
// into one contiguous range of stages per CTA.  192 threads: producer warp, MMA
// warp, four epilogue warps.  B's rows are the M side, so a lane is a column
// of D and a warp's stores of one row of D are contiguous at any alignment.
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 192;
constexpr double kStageUs = 0.3;
constexpr int kMaxSplit = 8;
constexpr int kSplitSumKb = 20;  // K = 2560

template <int BN>
struct SplitCfg {
    static constexpr int Q_BYTES = BN * kTileK;
    // two CTAs per SM, so that one's start and reduction overlap the other's loads: with
    // the whole shared memory for one CTA's ring, 160 tiles at 1 x 20480 x 5120 took
    // 28.9 us instead of 18.5
    static constexpr int STAGES = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
    static constexpr int SMEM = STAGES * (kPBytes + Q_BYTES + 2 * kSfBytes) + 1024 + 256;
    static constexpr int ACC = BN < 32 ? 32 : BN;
    static constexpr int TMEM = ACC <= 32 ? 64 : 2 * ACC;  // accumulator and two slots of 8 scale columns
    static_assert(2 * (SMEM + 1024) <= 233472 && 2 * TMEM <= 512, "two CTAs per SM");
    static_assert(STAGES * (kPBytes + Q_BYTES) >= BN * 128 * 4, "the ring holds the partial tile");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Four neighbours of one row of D.
__device__ __forceinline__ void store_four(const MxGemmArgs& p, int row, int col, const float4& v) {
    const float x[4] = {v.x, v.y, v.z, v.w};
    const int64_t at = static_cast<int64_t>(row) * p.ldd + col;
    const bool whole = col + 4 <= p.n;
    if (p.d_f32) {
        float* d = static_cast<float*>(p.d) + at;
        const bool vec = whole && (reinterpret_cast<uintptr_t>(d) & 15) == 0;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.accumulate) {
            if (vec) o = *reinterpret_cast<const float4*>(d);
            else o = make_float4(col < p.n ? d[0] : 0.f, col + 1 < p.n ? d[1] : 0.f, col + 2 < p.n ? d[2] : 0.f,
                                 col + 3 < p.n ? d[3] : 0.f);
        }
        const float y[4] = {p.accumulate ? o.x + x[0] : x[0], p.accumulate ? o.y + x[1] : x[1],
                            p.accumulate ? o.z + x[2] : x[2], p.accumulate ? o.w + x[3] : x[3]};
        if (vec) *reinterpret_cast<float4*>(d) = make_float4(y[0], y[1], y[2], y[3]);
        else
            for (int k = 0; k < 4; ++k)
                if (col + k < p.n) d[k] = y[k];
    } else {
        uint16_t* d = static_cast<uint16_t*>(p.d) + at;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
        const uint32_t w[2] = {*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)};
        if (whole && (reinterpret_cast<uintptr_t>(d) & 7) == 0) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
        else
            for (int k = 0; k < 4; ++k)
                if (col + k < p.n) d[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
}

// The sum of a cluster's CK parts: D's rows are dealt round-robin over the CTAs
// and their warps; a lane adds four columns, every part in rank order.  A warp
// takes 16 / CK rows at a time, so that each lane has 16 loads from the peers'
// shared memory in flight (with two rows at a time the latency of those loads
// made a split in two slower than none: 16.4 us against 14.5 at 355 x 3149 x
// 4704).
template <int CK, int EPI>
__device__ __forceinline__ void add_parts(const MxGemmArgs& p, float* part, int rank, int warp, int lane, int col0,
                                          int row0, int rows) {
    constexpr int U = 16 / CK;
    const uint32_t mine = smem_u32(part) + static_cast<uint32_t>(lane) * 16;
    const int col = col0 + lane * 4;
    const int step = CK * (kSplitThreads / 32);
    uint32_t from[CK];
#pragma unroll
    for (int k = 0; k < CK; ++k) from[k] = mapa_shared(mine, k);
    for (int c = rank + warp * CK; c < rows; c += U * step) {
        float4 x[U][CK];
#pragma unroll
        for (int h = 0; h < U; ++h)
#pragma unroll
            for (int k = 0; k < CK; ++k)
                if (c + h * step < rows) x[h][k] = ld_cluster_f4(from[k] + (c + h * step) * 512);
#pragma unroll
        for (int h = 0; h < U; ++h) {
            if (c + h * step >= rows || col >= p.n) continue;
            float4 v = x[h][0];
#pragma unroll
            for (int k = 1; k < CK; ++k)
                v = make_float4(v.x + x[h][k].x, v.y + x[h][k].y, v.z + x[h][k].z, v.w + x[h][k].w);
            // with an epilogue the sum goes over this CTA's own part, which only this lane reads
            if constexpr (EPI != kEpiNone) *reinterpret_cast<float4*>(part + (c + h * step) * 128 + lane * 4) = v;
            else store_four(p, row0 + c + h * step, col, v);
        }
    }
}

template <int BN, int EPI>
__global__ void __launch_bounds__(kSplitThreads, EPI ? 2 : 1)
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
    wait_for_earlier_kernels();
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
        int s = 0, slot = 0;
        uint32_t ph = 0;
        const uint32_t sfq_col = static_cast<uint32_t>(tq * BN % 128) / 32;  // A's rows inside its 128-row scale tile
        const uint64_t pd0 = desc_sw128(smem_u32(sp)), qd0 = desc_sw128(smem_u32(sq)), sd0 = desc_sf(smem_u32(ssf));
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), ph, p.err, bail))) break;
            tc_fence_after();
            const uint32_t tsf = tmem + C::ACC + slot * 8;
            const uint64_t pd = pd0 + static_cast<uint64_t>(s * (kPBytes >> 4));
            const uint64_t qd = qd0 + static_cast<uint64_t>(s * (C::Q_BYTES >> 4));
            const uint64_t sd = sd0 + static_cast<uint64_t>(s * (2 * kSfBytes >> 4));
            const int nk = kb + 1 < p.num_kb ? 4 : p.last_nk;
            if (elect_one()) {
                tmem_cp_sf(tsf, sd);
                tmem_cp_sf(tsf + 4, sd + (kSfBytes >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    if (kk < nk)
                        umma_mx(tmem, pd + 2 * kk, qd + 2 * kk, mx_idesc(kTileP, BN) | sf_id(kk), tsf, tsf + 4 + sfq_col,
                                (kb - kb0) | kk);
                umma_commit(smem_u32(&empty[s]));
            }
            __syncwarp();
            slot ^= 1;
            if (++s == C::STAGES) { s = 0; ph ^= 1u; }
        }
        // also covers every MMA issued before an early exit
        if (elect_one()) {
            if (!p.inject) umma_commit(smem_u32(tfull));
            mbar_wait(smem_u32(tfull), 0, p.err, bail, false);
        }
    }
    __syncwarp();
    // the epilogue warps wait for the accumulator; the others only join the barriers below
    const int q = warp & 3;
    const int col = tp * kTileP + q * 32 + lane;  // column of D
    const int row0 = tq * BN;
    const int rows = min(BN, p.m - row0);
    EpiPiece<EPI, true, true> piece;
    float2 bias[4];
    if (EPI && ck == 1 && warp >= 2) {
        piece.bias(p, col - lane, bias);
        piece.load(p, row0, col - lane);
    }
    if (warp >= 2) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(tfull), 0, p.err, bail));
        tc_fence_after();
        if (EPI && ok && ck == 1) {
            // the ring has been read: it turns the pieces
            float* stage = reinterpret_cast<float*>(smem) + q * (kPieceBytes / 4);
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += kPieceRows) {
                piece.begin(p, row0 + c0, col - lane);
                uint32_t r[16];
                __syncwarp();
                tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, r);
                tmem_ld_wait();
                tmem_ld_pin16(r);
                EpiPiece<EPI, true, true> ahead;
                if (c0 + kPieceRows < rows) ahead.load(p, row0 + c0 + kPieceRows, col - lane);
                piece.finish(p, stage, row0 + c0, col - lane, bias, r);
                piece.take(p, ahead);
            }
        } else if (ok) {
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += 32) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0, r);
                tmem_ld_wait();
                tmem_ld_pin(r);
                if (ck == 1) {
                    store_chunk(p, col, row0 + c0, r);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j >= rows) break;
                    part[(c0 + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
                }
            }
        }
        tc_fence_before();
    }
    if (ck > 1) {
        __syncwarp();
        cluster_sync_all();
        const int c0 = tp * kTileP;
        switch (ck) {
            case 2: add_parts<2, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            case 3: add_parts<3, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            case 4: add_parts<4, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            case 5: add_parts<5, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            case 6: add_parts<6, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            case 7: add_parts<7, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
            default: add_parts<8, EPI>(p, part, rank, warp, lane, c0, row0, rows); break;
        }
        if constexpr (EPI != kEpiNone) {
            // the same rows and columns as above, one copy of the epilogue's code
            const int at = c0 + lane * 4, count = p.n - at;
            float b4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) b4[k] = p.e.bias && k < count ? p.e.bias[at + k] : 0.f;
            const int step = ck * (kSplitThreads / 32);
            EpiRow<EPI == kEpiF32 || EPI == kEpiF32Any, EPI == kEpiBf16 || EPI == kEpiF32> now, ahead;
            int c = rank + warp * ck;
            if (c < rows) now.load(p, row0 + c, at, count);
#pragma unroll 1
            for (; c < rows; c += step) {
                if (c + step < rows) ahead.load(p, row0 + c + step, at, count);
                if (count > 0) {
                    const float4 v = *reinterpret_cast<const float4*>(part + c * 128 + lane * 4);
                    const float2 z[2] = {make_float2(v.x + b4[0], v.y + b4[1]), make_float2(v.z + b4[2], v.w + b4[3])};
                    now.finish(p, row0 + c, at, count, z);
                }
                now = ahead;
            }
        }
        __syncwarp();
        cluster_arrive_relaxed();  // a CTA's part stays until its peers have read it
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// K = 0: the sum is empty (and D unchanged when accumulating: no launch).
__global__ void __launch_bounds__(256) mx_gemm_zero_kernel(const __grid_constant__ MxGemmArgs p) {
    wait_for_earlier_kernels();
    const int64_t total = static_cast<int64_t>(p.m) * p.n;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll)
        if (p.d_f32) static_cast<float*>(p.d)[i / p.n * p.ldd + i % p.n] = 0.f;
        else static_cast<uint16_t*>(p.d)[i / p.n * p.ldd + i % p.n] = 0u;
}

// The same with an epilogue: z = 0 before the bias.
template <bool F32>
__global__ void __launch_bounds__(256) mx_gemm_empty_kernel(const __grid_constant__ MxGemmArgs p) {
    wait_for_earlier_kernels();
    const int64_t total = static_cast<int64_t>(p.m) * p.n;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int row = static_cast<int>(i / p.n), col = static_cast<int>(i % p.n);
        EpiRow<F32, false> x;
        x.load(p, row, col, 1);
        const float2 z[2] = {make_float2(p.e.bias ? p.e.bias[col] : 0.f, 0.f), make_float2(0.f, 0.f)};
        x.finish(p, row, col, 1, z);
    }
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

// Tiled scales of `rows` rows as [row tiles][num_kb][128 words]: boxes of `tiles`
// 512-byte scale tiles of one K stage, zero past the last row tile.
bool map_scales(CUtensorMap* m, const uint8_t* base, int num_kb, int64_t rows, int tiles) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(num_kb), static_cast<cuuint64_t>((rows + 127) / 128)};
    const cuuint64_t strides[2] = {kSfBytes, static_cast<cuuint64_t>(num_kb) * kSfBytes};
    const cuuint32_t box[3] = {128, 1, static_cast<cuuint32_t>(tiles)};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `size` CTAs, set up while the kernel before drains (launch_early's rule).
void cluster_early(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int size) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

template <int BN>
void split_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int tiles_p, int tiles_q, int split, cudaStream_t st) {
    cfg = {};
    cfg.gridDim = dim3(tiles_p * split, tiles_q, 1);
    cfg.blockDim = dim3(kSplitThreads, 1, 1);
    cfg.dynamicSmemBytes = SplitCfg<BN>::SMEM;
    cfg.stream = st;
    cluster_early(cfg, attr, split);
}

// Clusters of `split` CTAs that run at once, asked once per device.  The query counts
// one CTA per SM for a kernel that allocates TMEM (152, 76, 36 and 15 clusters of 1, 2,
// 4 and 8); two were seen to run (40 clusters of 4 in the time of one round).
template <int BN>
int resident_clusters(int split) {
    static std::atomic<int> cached[64][kMaxSplit + 1];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool keep = dev >= 0 && dev < 64;
    if (keep && cached[dev][split].load(std::memory_order_relaxed)) return cached[dev][split].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    split_config<BN>(cfg, attr, 1, 1, split, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_split_kernel<BN, kEpiNone>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, device_sm_count() / (2 * split));
    }
    n *= 2;
    if (keep) cached[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs of a cluster that share a tile's K, and the estimated time in us: rounds of
// resident clusters x stages x the time of a stage, and the addition of the parts.
// Measured: a stage takes 0.3 us in a CTA that has its SM to itself (128 x 128 tiles,
// 37 stages in 11.4 us; 128 x 16, 40 in 11.1), 0.45 us where two share an SM, or
// what the CTAs get of B from HBM together; adding 128 rows of parts takes 4.5 us, one
// row 0.7; a round starts and ends in 3.  With an epilogue 2 more, and 0.5 for each 16 rows of
// an undivided tile, which four warps finish (divided ones are finished by six warps of
// each CTA): 301 x 1408 x 2048 bf16 with GELU 11.6 us in whole tiles of 128, 8.8 in tiles of 64
// with K in four parts.
template <int BN>
int split_for(int tiles_p, int tiles_q, const MxGemmArgs& p, double* cost) {
    const int rows = p.m, num_kb = p.num_kb;
    const double bytes = kPBytes + SplitCfg<BN>::Q_BYTES + 2 * kSfBytes;
    const int64_t tiles = static_cast<int64_t>(tiles_p) * tiles_q;
    // fp32 D: no part sums more than kSplitSumKb stages (the truncation that SUMS is about)
    const int least = p.d_f32 ? std::min(kMaxSplit, (num_kb + kSplitSumKb - 1) / kSplitSumKb) : 1;
    int best = 0;
    for (int s = least; s <= kMaxSplit && s <= num_kb; ++s) {
        const int cap = resident_clusters<BN>(s);
        const double ctas = static_cast<double>(std::min<int64_t>(tiles, cap) * s);
        const double stage = std::max({kStageUs, bytes * std::ceil(ctas / device_sm_count()) / 0.15e6,
                                       (kPBytes + kSfBytes) * ctas / tiles_q / 6.5e6});
        const double rounds = static_cast<double>((tiles + cap - 1) / cap);
        const double c = rounds * (((num_kb + s - 1) / s) * stage + 3.0 + (s > 1 ? 0.7 + 0.03 * std::min(rows, BN) : 0.0) +
                                   (p.epilogue ? 2.0 + (s > 1 ? 0.0 : 0.5 * ((std::min(rows, BN) + kPieceRows - 1) / kPieceRows)) : 0.0));
        if (!best || c < *cost) *cost = c, best = s;
    }
    return best;
}

// The split kernel with BN rows of A per tile: its parts and what they are estimated to take.
template <int BN>
cudaError_t split_form(const MxGemmArgs& p, MxGemmForm* f, double* cost) {
    static PerDevice done;
    const cudaError_t e = allow_smem(mx_gemm_split_kernel<BN, kEpiNone>, SplitCfg<BN>::SMEM, done);  // before its occupancy is asked
    if (e != cudaSuccess) return e;
    f->tile = BN;
    f->parts = split_for<BN>((p.n + kTileP - 1) / kTileP, (p.m + BN - 1) / BN, p, cost);
    f->sums = 0;
    return cudaSuccess;
}

// Tiles of 128 rows, or with an epilogue of 64 where those are estimated to take less: there
// are then twice as many warps to finish them.  (Tiles start at multiples of 64 rows:
// a tile's scales begin at an even column of TMEM.)
cudaError_t split_few_rows(const MxGemmArgs& p, MxGemmForm* f, double* cost) {
    const cudaError_t e = split_form<128>(p, f, cost);
    if (e != cudaSuccess || !p.epilogue || (p.m + 63) / 64 > 65535) return e;
    MxGemmForm g;
    double c;
    const cudaError_t e64 = split_form<64>(p, &g, &c);
    if (e64 == cudaSuccess && c < *cost) *f = g, *cost = c;
    return e64;
}

template <int BN>
cudaError_t launch_split(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, const MxGemmArgs& p, cudaStream_t st) {
    CUtensorMap ma, mb;
    if (!map_codes(&ma, a, p.k, p.m, lda, BN) || !map_codes(&mb, b, p.k, p.n, ldb, kTileP)) return cudaErrorUnknown;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    split_config<BN>(cfg, attr, (p.n + kTileP - 1) / kTileP, (p.m + BN - 1) / BN, p.split, st);
    auto kernel = mx_gemm_split_kernel<BN, kEpiNone>;
    if (p.epilogue) {
        static PerDevice done[5];
        kernel = p.epilogue == kEpiBf16  ? mx_gemm_split_kernel<BN, kEpiBf16>
                 : p.epilogue == kEpiF32 ? mx_gemm_split_kernel<BN, kEpiF32>
                 : p.d_f32               ? mx_gemm_split_kernel<BN, kEpiF32Any>
                                         : mx_gemm_split_kernel<BN, kEpiBf16Any>;
        const cudaError_t e = allow_smem(kernel, SplitCfg<BN>::SMEM, done[p.epilogue]);
        if (e != cudaSuccess) return e;
    }
    note_launch();
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
}

template <int BN, bool SUMS, int EPI = kEpiNone>
cudaError_t launch_pair(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, MxGemmArgs p, cudaStream_t st) {
    using C = PairMx<BN>;
    if constexpr (EPI == kEpiNone) {
        if constexpr (BN < 256) {
            if (p.epilogue == kEpiF32) return launch_pair<BN, SUMS, kEpiF32>(a, lda, b, ldb, p, st);
            if (p.epilogue == kEpiF32Any) return launch_pair<BN, SUMS, kEpiF32Any>(a, lda, b, ldb, p, st);
        }
        if constexpr (!SUMS) {
            if (p.epilogue == kEpiBf16) return launch_pair<BN, SUMS, kEpiBf16>(a, lda, b, ldb, p, st);
            if (p.epilogue == kEpiBf16Any) return launch_pair<BN, SUMS, kEpiBf16Any>(a, lda, b, ldb, p, st);
        }
        // mx_gemm_form names no other tile; D without its epilogue would look like a result
        if (p.epilogue) return cudaErrorInvalidValue;
    }
    constexpr int smem = C::SMEM + (EPI ? kPairEpiWarps * kPieceBytes : 0);
    static_assert(smem <= 232448, "the ring and the pieces");
    static PerDevice done;
    cudaError_t e = allow_smem(mx_gemm_pair_kernel<BN, SUMS, EPI>, smem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mp, mq, msp, msq;
    if (!map_codes(&mp, b, p.k, p.n, ldb, kTileP) || !map_codes(&mq, a, p.k, p.m, lda, BN / 2) ||
        !map_scales(&msp, p.sb, p.num_kb, p.n, 1) || !map_scales(&msq, p.sa, p.num_kb, p.m, C::NSF))
        return cudaErrorUnknown;
    p.tiles_p = (p.n + 255) / 256;
    p.tiles_q = (p.m + BN - 1) / BN;
    const int64_t total = static_cast<int64_t>(p.tiles_p) * p.tiles_q;
    const int pairs = static_cast<int>(total < device_sm_count() / 2 ? total : device_sm_count() / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cluster_early(cfg, attr, 2);
    note_launch();
    return cudaLaunchKernelEx(&cfg, mx_gemm_pair_kernel<BN, SUMS, EPI>, mp, mq, msp, msq, p);
}

}  // namespace

// k > 0.  The kernel, its tile width, the split of K and whether K is summed in chunks.
cudaError_t mx_gemm_form(const MxGemmArgs& args, MxGemmForm* f) {
    MxGemmArgs p = args;
    p.num_kb = (p.k + kTileK - 1) / kTileK;
    double cost;
    // fp32 D over a K that eight parts of kSplitSumKb stages do not cover: the pair kernel's
    // sums, however few the rows (5 x 5120: K = 20480 in eight parts 22.2 us, 24576 on
    // pairs 52.5)
    const bool long_sum = p.d_f32 && p.num_kb > kMaxSplit * kSplitSumKb;
    if (!long_sum) {
        if (p.m <= 16) return split_form<16>(p, f, &cost);
        if (p.m <= 32) return split_form<32>(p, f, &cost);
        if (p.m <= 64) return split_form<64>(p, f, &cost);
        if (p.m <= 128) return split_few_rows(p, f, &cost);
    }
    // The tile width that leaves the least time to the pair with the most tiles.  A
    // stage's time goes with the rows it loads (256 + BN): 128-wide tiles took 0.79 of
    // the time of 256-wide ones (293 and 371 ns per stage, K = 5120, 640 tiles of 256);
    // a tile's epilogue takes about 2.2 us, filling and emptying the pipeline 4.
    // With sums at most 192: a thread of the eight epilogue warps would hold 128 of
    // them at 256, and ten warps leave it 168 registers (192 takes all, 28 bytes spilled).
    const bool sums = p.d_f32 && p.num_kb > kChunkK / kTileK;
    // With an epilogue and fp32 D the products of K <= kChunkK take less than their epilogue,
    // and 128 rows finish as fast as half of 256.
    const bool wide_never = p.d_f32 && p.epilogue;
    const int64_t pairs = device_sm_count() / 2;
    int best = 0;
    double least = 0;
    for (const int bn : {256, 192, 128}) {
        if (bn > 192 && (sums || wide_never)) continue;
        const int64_t tiles = static_cast<int64_t>((p.n + 255) / 256) * ((p.m + bn - 1) / bn);
        // An epilogue (hm_epilogue) takes 1 us per 32 rows, and the last tile's overlaps nothing; a
        // stage of 512 rows 0.30 us where no power cap holds it down.  With these every form of
        // 300 x 5120 x 5120, 512 x 20480 x 5120, 777 x 2048 x 1408, 1024 x 4096 x 4096, 2048 x 2048 x
        // 1024 and 4096 x 4096 x 1024 bf16 is the fastest one measured or within 3 % of it
        // (1024 x 4096 x 4096 with GELU: 19.6 us on 256-row pairs, 21.5 in whole 128-row tiles).
        const double stage = p.epilogue ? 0.30 / 512 : 0.37 / 512;
        const double sum = p.num_kb * (256 + bn) * stage, last = p.epilogue ? bn / 32 * 1.0 : 2.2;
        const double c = static_cast<double>((tiles + pairs - 1) / pairs) * std::max(sum, last) + 4.0 + (p.epilogue ? std::min(sum, last) : 0.0);
        if (!best || c < least) best = bn, least = c;
    }
    // Too few tiles for the pairs: 128 x 128 tiles with K split over clusters.  Both
    // forms measured for 129 to 1024 rows at n x k = 5120 x 5120, 20480 x 5120,
    // 4096 x 4096 and 1408 x 2048, bf16 and fp32 D: the chosen one is the faster or
    // within 4 % of it (129 x 5120 x 5120 bf16 12.4 us split, 14.1 on pairs; 512 rows 17.1
    // and 15.5), but for 300 and 384 x 20480 x 5120 bf16, where two rounds of
    // undivided tiles take 48 us that the estimate puts at 42, and pairs 38.
    if ((static_cast<int64_t>(p.m) + 127) / 128 <= 65535 && !long_sum) {
        const cudaError_t e = split_few_rows(p, f, &cost);
        if (e != cudaSuccess || cost < least) return e;
    }
    f->tile = best;
    f->parts = 0;
    f->sums = sums;
    return cudaSuccess;
}

cudaError_t launch_mx_gemm(const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, const MxGemmArgs& args,
                           cudaStream_t st) {
    MxGemmArgs p = args;
    if (p.epilogue) {
        const int64_t es = p.d_f32 ? 4 : 2;
        const auto rows16 = [&](const void* q, int64_t ld) { return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * es % 16 == 0); };
        const bool vec = p.n % 8 == 0 && rows16(p.d, p.ldd) && rows16(p.e.in, p.e.ld_in) && rows16(p.e.in2, p.e.ld_in2) && rows16(p.e.out2, p.e.ld_out2);
        p.epilogue = p.d_f32 ? (vec ? kEpiF32 : kEpiF32Any) : (vec ? kEpiBf16 : kEpiBf16Any);
    }
    if (p.k == 0) {
        if (p.accumulate) return cudaSuccess;
        const int64_t blocks = (static_cast<int64_t>(p.m) * p.n + 255) / 256;
        note_launch();
        if (p.epilogue) {
            const auto kernel = p.d_f32 ? mx_gemm_empty_kernel<true> : mx_gemm_empty_kernel<false>;
            kernel<<<resident_grid(kernel, 256, blocks), 256, 0, st>>>(p);
            return cudaGetLastError();
        }
        mx_gemm_zero_kernel<<<resident_grid(mx_gemm_zero_kernel, 256, blocks), 256, 0, st>>>(p);
        return cudaGetLastError();
    }
    p.num_kb = (p.k + kTileK - 1) / kTileK;
    p.last_nk = (p.k - (p.num_kb - 1) * kTileK) / 32;
    p.err = device_error_word();
    p.inject = inject_mx_timeout();
    MxGemmForm f;
    const cudaError_t e = mx_gemm_form(p, &f);
    if (e != cudaSuccess) return e;
    p.split = f.parts;
    if (f.parts) {
        if (f.tile == 16) return launch_split<16>(a, lda, b, ldb, p, st);
        if (f.tile == 32) return launch_split<32>(a, lda, b, ldb, p, st);
        if (f.tile == 64) return launch_split<64>(a, lda, b, ldb, p, st);
        return launch_split<128>(a, lda, b, ldb, p, st);
    }
    if (f.tile == 256) return launch_pair<256, false>(a, lda, b, ldb, p, st);
    if (f.tile == 192) return f.sums ? launch_pair<192, true>(a, lda, b, ldb, p, st) : launch_pair<192, false>(a, lda, b, ldb, p, st);
    return f.sums ? launch_pair<128, true>(a, lda, b, ldb, p, st) : launch_pair<128, false>(a, lda, b, ldb, p, st);
}

}  // namespace hm
