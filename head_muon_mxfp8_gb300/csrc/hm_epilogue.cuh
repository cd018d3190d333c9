// Epilogue of the MXFP8 product with bias, activation, gate, residual and their
// gradients (hm_epilogue), for the kernels of hm_mxgemm.cu.
//
// An accumulator's chunk comes out of TMEM with a lane per column of D.  16 rows x 32
// columns of a warp are one piece.  Where all matrices have 16-byte rows, the piece
// turns through shared memory, so that a lane holds 8 neighbours of two rows and
// every matrix is read and written 16 bytes at a time; with an element per lane and
// instruction instead, the epilogue without any activation issued 30 instructions per
// element and took 12 us of a 256 x 256 tile whose products take 3.3 (4096 x
// 4096 x 1024 bf16: 48.6 us against 17.7 plain; with bias, GELU and the kept sum 81.5, now
// 32).  Otherwise a lane keeps its column, whose neighbours' accesses coalesce at any
// alignment (36 us there; both of a gated pair's gradients 56 against 47).
// What a piece reads is loaded one piece ahead, or, by a lane that keeps its column (twice
// the registers), before the piece's accumulators are waited for.
//
// Under the power cap a large product pays for every instruction of its epilogue, so
// one branch on form and activation leads to straight code up to its stores (values
// that several branches hand on cost a move each), arithmetic goes two elements at a
// time (f32x2), and exponentials and quotients are the hardware's: exp2 within 2^-22,
// 1 / y within 2^-23, on a sum that is rounded to fp32 anyway.
#pragma once

#include "hm.h"
#include "hm_ops.h"
#include "hm_vec.cuh"

namespace hm {

constexpr int kPieceRows = 16;
constexpr int kPiecePitch = 36;  // floats: rows 4 banks apart
constexpr int kPieceBytes = kPieceRows * kPiecePitch * 4;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float inv_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 exp2_fast(float2 x) { return make_float2(exp2_fast(x.x), exp2_fast(x.y)); }
__device__ __forceinline__ float2 inv_fast(float2 x) { return make_float2(inv_fast(x.x), inv_fast(x.y)); }

// Activations of two elements: value() and both(), with the slope.
constexpr float kLog2e = 1.4426950408889634f;
// max(x, 0), and x itself where `cut` is NaN; a NaN stays.
struct ActCut {
    float cut;
    __device__ __forceinline__ float2 value(float2 x) const { return make_float2(x.x <= cut ? 0.f : x.x, x.y <= cut ? 0.f : x.y); }
    __device__ __forceinline__ float2 both(float2 x, float2& slope) const {
        slope = make_float2(x.x <= cut ? 0.f : 1.f, x.y <= cut ? 0.f : 1.f);
        return value(x);
    }
};
// x s(x), s(x) = 1 / (1 + exp(-x)); slope s + x s (1 - s)
struct ActSilu {
    __device__ __forceinline__ float2 s(float2 x) const { return inv_fast(add2(exp2_fast(mul2(x, both2(-kLog2e))), both2(1.f))); }
    __device__ __forceinline__ float2 value(float2 x) const { return mul2(x, s(x)); }
    __device__ __forceinline__ float2 both(float2 x, float2& slope) const {
        const float2 t = s(x), f = mul2(x, t);
        slope = fma2(f, fma2(t, both2(-1.f), both2(1.f)), t);
        return f;
    }
};
// GELU's tanh form is x s(u), u = x (c0 + c1 x^2), as 0.5 (1 + tanh(w)) = s(2 w); slope
// s + x s (1 - s) u', where a u' that left fp32 must not meet a vanished s (1 - s).
struct ActGeluTanh {
    static constexpr float c0 = 1.5957691216057308f, c1 = 0.0713548162726009f;  // 2 sqrt(2 / pi), 0.044715 of it
    __device__ __forceinline__ float2 s(float2 x, float2 x2) const {
        const float2 w = mul2(x, fma2(x2, both2(-kLog2e * c1), both2(-kLog2e * c0)));
        return inv_fast(add2(exp2_fast(w), both2(1.f)));
    }
    __device__ __forceinline__ float2 value(float2 x) const { return mul2(x, s(x, mul2(x, x))); }
    __device__ __forceinline__ float2 both(float2 x, float2& slope) const {
        const float2 x2 = mul2(x, x), t = s(x, x2), f = mul2(x, t);
        const float2 du = fma2(make_float2(fminf(x2.x, 1e30f), fminf(x2.y, 1e30f)), both2(3.f * c1), both2(c0));
        slope = fma2(mul2(f, fma2(t, both2(-1.f), both2(1.f))), du, t);
        return f;
    }
};
// x Phi(x); slope Phi(x) + x phi(x).  Phi(-|x|) = t q(t) exp(-x^2 / 2) with t = 1 / (1 + p |x|):
// small values come from products alone, where 1 + erf loses them to cancellation (all of
// them below x = -5.6).  q is a polynomial with a small largest error of Phi, relative to it, down
// to x = -13.6, where the exponential leaves the normal numbers.
//   fp32 results: p = 0.3, degree 9, least squares weighted towards the largest relative error:
//     2^-28; with all roundings (18 + 1.1 x^2) 2^-24 of Phi.
//   bf16 results: p = 0.292, degree 5, the largest error in units of min(2e-7, 2^-13 Phi) by linear
//     programming: 0.7e-7 and 2^-14.5 of Phi, a hundredth of bf16's half step.
// The exponential is the slope's too.  (fp32, 4096 x 4096 x 1024: 40.0 us; by CUDA's erfcf 54.3, by its
// erff, which cancels, 45.5.)
template <bool F32>
struct ActGelu {
    static __device__ __forceinline__ float2 series(float2 t) {
        if constexpr (F32) {
            float2 q = fma2(t, both2(-0.0205989908f), both2(0.112297878f));
            q = fma2(q, t, both2(-0.227877095f));
            q = fma2(q, t, both2(0.191316977f));
            q = fma2(q, t, both2(-0.0790171549f));
            q = fma2(q, t, both2(0.0959282517f));
            q = fma2(q, t, both2(0.0784726888f));
            q = fma2(q, t, both2(0.110216685f));
            q = fma2(q, t, both2(0.119574197f));
            q = fma2(q, t, both2(0.119686566f));
            return q;
        } else {
            float2 q = fma2(t, both2(-0.0865621045f), both2(0.27013579f));
            q = fma2(q, t, both2(-0.0754651725f));
            q = fma2(q, t, both2(0.170437515f));
            q = fma2(q, t, both2(0.104019143f));
            q = fma2(q, t, both2(0.117434815f));
            return q;
        }
    }
    __device__ __forceinline__ float2 phi(float2 x, float2 g) const {
        const float2 t = inv_fast(fma2(make_float2(fabsf(x.x), fabsf(x.y)), both2(F32 ? 0.3f : 0.292f), both2(1.f)));
        const float2 q = mul2(mul2(series(t), t), g);
        return make_float2(x.x < 0.f ? q.x : 1.f - q.x, x.y < 0.f ? q.y : 1.f - q.y);
    }
    __device__ __forceinline__ float2 g(float2 x) const { return exp2_fast(mul2(mul2(x, x), both2(-0.5f * kLog2e))); }
    __device__ __forceinline__ float2 value(float2 x) const { return mul2(x, phi(x, g(x))); }
    __device__ __forceinline__ float2 both(float2 x, float2& slope) const {
        const float2 e = g(x), p = phi(x, e);
        slope = fma2(mul2(x, both2(0.39894228040143268f)), e, p);
        return mul2(x, p);
    }
};

// D and out2 of P pairs, handed to store(D, out2).  z: the product with the bias; x: in;
// y: in2.
template <int P, class Act, class Store>
__device__ __forceinline__ void finish_as(const MxEpilogue& e, const Act act, const float2 (&z)[P], const float2 (&x)[P],
                                          const float2 (&y)[P], const Store& store) {
    float2 d[P], w[P];
    if (e.form == HM_EPI_FORWARD) {
        if (e.in) {
#pragma unroll
            for (int j = 0; j < P; ++j) d[j] = add2(act.value(z[j]), x[j]);
            store(d, z);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) d[j] = act.value(z[j]);
            store(d, z);
        }
    } else if (e.form == HM_EPI_GATED) {
#pragma unroll
        for (int j = 0; j < P; ++j) d[j] = mul2(z[j], act.value(x[j]));
        store(d, z);
    } else if (e.form == HM_EPI_GRADIENT) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float2 slope;
            act.both(x[j], slope);
            d[j] = mul2(z[j], slope);
        }
        store(d, z);
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            float2 slope;
            d[j] = mul2(z[j], act.both(x[j], slope));
            w[j] = mul2(mul2(z[j], y[j]), slope);
        }
        store(d, w);
    }
}
// Calls f(activation).
template <bool F32, class F>
__device__ __forceinline__ void with_activation(int act, const F& f) {
    if (act <= HM_ACT_RELU) {
        f(ActCut{act == HM_ACT_RELU ? 0.f : __int_as_float(0x7fffffff)});
    } else if (act == HM_ACT_GELU) {
        f(ActGelu<F32>{});
    } else if (act == HM_ACT_GELU_TANH) {
        f(ActGeluTanh{});
    } else {
        f(ActSilu{});
    }
}
template <bool F32, int P, class Store>
__device__ __forceinline__ void finish_elements(const MxEpilogue& e, const float2 (&z)[P], const float2 (&x)[P],
                                                const float2 (&y)[P], const Store& store) {
    with_activation<F32>(e.act, [&](const auto act) { finish_as<P>(e, act, z, x, y, store); });
}
// The same in little code, for the kernels whose time is not their epilogue's: the
// activation and its slope first, then the form.
template <bool F32, int P, class Store>
__device__ __forceinline__ void finish_short(const MxEpilogue& e, const float2 (&z)[P], const float2 (&x)[P],
                                             const float2 (&y)[P], const Store& store) {
    const bool forward = e.form == HM_EPI_FORWARD;
    float2 f[P], slope[P], w[P];
#pragma unroll
    for (int j = 0; j < P; ++j) f[j] = forward ? z[j] : x[j], w[j] = z[j];
    with_activation<F32>(e.act, [&](const auto act) {
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = act.both(f[j], slope[j]);
    });
    if (forward) {
        if (e.in)
#pragma unroll
            for (int j = 0; j < P; ++j) f[j] = add2(f[j], x[j]);
    } else {
        const bool plain = e.form == HM_EPI_GRADIENT;
        if (e.form == HM_EPI_GATED_GRADIENT)
#pragma unroll
            for (int j = 0; j < P; ++j) w[j] = mul2(mul2(w[j], y[j]), slope[j]);
#pragma unroll
        for (int j = 0; j < P; ++j) f[j] = mul2(z[j], plain ? slope[j] : f[j]);
    }
    store(f, w);
}

template <bool F32, int N, int P>
__device__ __forceinline__ void to_pairs(const RowVec<F32, N>& v, float2 (&x)[P], int at) {
    float t[N];
    v.get(t);
#pragma unroll
    for (int j = 0; j < N; j += 2) x[at + j / 2] = make_float2(t[j], t[j + 1]);
}
template <bool F32, int N, int P>
__device__ __forceinline__ RowVec<F32, N> from_pairs(const float2 (&x)[P], int at) {
    float t[N];
#pragma unroll
    for (int j = 0; j < N; j += 2) t[j] = x[at + j / 2].x, t[j + 1] = x[at + j / 2].y;
    RowVec<F32, N> v;
    v.set(t);
    return v;
}

// Four neighbours of one row, `count` of them inside D (<= 0: none); VEC: whole and aligned.
template <bool F32, bool VEC>
struct EpiRow {
    RowVec<F32, 4> in, in2;
    __device__ __forceinline__ void load(const MxGemmArgs& p, int row, int col, int count) {
        if (p.e.in) fetch(in, p.e.in, row * p.e.ld_in + col, count);
        if (p.e.in2) fetch(in2, p.e.in2, row * p.e.ld_in2 + col, count);
    }
    static __device__ __forceinline__ void fetch(RowVec<F32, 4>& v, const void* base, int64_t at, int count) {
        if (!VEC) v.load_some(base, at, count);
        else if (count > 0) v.load(base, at);
    }
    static __device__ __forceinline__ void put(const RowVec<F32, 4>& v, void* base, int64_t at, int count) {
        if (!VEC) v.store_some(base, at, count);
        else v.store(base, at);
    }
    __device__ __forceinline__ void finish(const MxGemmArgs& p, int row, int col, int count, const float2 (&z)[2]) const {
        float2 x[2], y[2];
        to_pairs<F32, 4>(in, x, 0);
        to_pairs<F32, 4>(in2, y, 0);
        finish_short<F32>(p.e, z, x, y, [&](const float2(&d)[2], const float2(&w)[2]) {
            if (p.e.out2) put(from_pairs<F32, 4>(w, 0), p.e.out2, row * p.e.ld_out2 + col, count);
            put(from_pairs<F32, 4>(d, 0), p.d, row * p.ldd + col, count);
        });
    }
};

// Which epilogue a kernel has: on bf16 or fp32 matrices, whose rows are 16-byte aligned
// and a multiple of 8 elements long, or not.
constexpr int kEpiNone = 0, kEpiBf16 = 1, kEpiF32 = 2, kEpiBf16Any = 3, kEpiF32Any = 4;

// Pieces of a warp.  AHEAD: load() one piece ahead of its finish() (aligned rows only);
// otherwise finish() loads what it needs itself, but for a lane's column: begin() does.
// SHORT: finish_short.
template <int EPI, bool AHEAD, bool SHORT>
struct EpiPiece {
    static constexpr bool F32 = EPI == kEpiF32 || EPI == kEpiF32Any, VEC = EPI == kEpiBf16 || EPI == kEpiF32;
    static constexpr bool kAhead = AHEAD && VEC;
    RowVec<F32, 8> in[2], in2[2];                      // VEC: rows lane / 4 and 8 more, columns 8 (lane % 4) ..
    RowVec<F32, 1> cin[VEC ? 1 : 16], cin2[VEC ? 1 : 16];  // else: the lane's column

    __device__ __forceinline__ void load_one(const MxGemmArgs& p, int h, int row, int col) {
        if (row >= p.m || col >= p.n) return;
        in[h].load(p.e.in, row * p.e.ld_in + col);
        if (p.e.in2) in2[h].load(p.e.in2, row * p.e.ld_in2 + col);
    }
    __device__ __forceinline__ void load(const MxGemmArgs& p, int row0, int col0) {
        if (!kAhead || !p.e.in) return;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int h = 0; h < 2; ++h) load_one(p, h, row0 + (lane >> 2) + 8 * h, col0 + (lane & 3) * 8);
    }
    static __device__ __forceinline__ void column(RowVec<F32, 1> (&v)[VEC ? 1 : 16], const void* base, int64_t ld, int64_t at, int rows) {
        const char* q = static_cast<const char*>(base) + at * (F32 ? 4 : 2);
        const int64_t step = ld * (F32 ? 4 : 2);
        if (rows >= 16) {
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 16); ++j, q += step) v[j].load(q, 0);
        } else {
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 16); ++j, q += step)
                if (j < rows) v[j].load(q, 0);
        }
    }
    __device__ __forceinline__ void begin(const MxGemmArgs& p, int row0, int col0) {
        const int col = col0 + (threadIdx.x & 31);
        if (VEC || !p.e.in || col >= p.n) return;
        column(cin, p.e.in, p.e.ld_in, row0 * p.e.ld_in + col, p.m - row0);
        if (p.e.in2) column(cin2, p.e.in2, p.e.ld_in2, row0 * p.e.ld_in2 + col, p.m - row0);
    }
    __device__ __forceinline__ void take(const MxGemmArgs& p, const EpiPiece& next) {
        if (kAhead && p.e.in) *this = next;
    }
    // Bias of the columns that this lane finishes: 8, or one.
    static __device__ __forceinline__ void bias(const MxGemmArgs& p, int col0, float2 (&b)[4]) {
        const int lane = threadIdx.x & 31, first = VEC ? col0 + (lane & 3) * 8 : col0 + lane;
        const auto at = [&](int k) { return p.e.bias && first + k < p.n ? p.e.bias[first + k] : 0.f; };
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = VEC ? make_float2(at(2 * k), at(2 * k + 1)) : both2(k ? 0.f : at(0));
    }
    // Rows row0 .. row0 + 15, columns col0 .. col0 + 31 of D; r: the lane's column of the
    // accumulator; stage: kPieceBytes of the warp's own.
    __device__ __forceinline__ void finish(const MxGemmArgs& p, float* stage, int row0, int col0, const float2 (&b)[4],
                                           const uint32_t (&r)[16]) {
        const int lane = threadIdx.x & 31;
        if constexpr (VEC) {
            __syncwarp();  // the piece before has been read
#pragma unroll
            for (int j = 0; j < 16; ++j) stage[j * kPiecePitch + lane] = __uint_as_float(r[j]);
            __syncwarp();
            const int col = col0 + (lane & 3) * 8, r0 = row0 + (lane >> 2);
            const float* mine = stage + (lane >> 2) * kPiecePitch + (lane & 3) * 8;
            if (col >= p.n || r0 >= p.m) return;
            // bf16: both rows in one go; fp32: one after the other, for the registers
            constexpr int H = F32 ? 1 : 2;
#pragma unroll 1
            for (int h0 = 0; h0 < 2; h0 += H) {
                float2 z[4 * H], x[4 * H], y[4 * H];
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    const float4* s = reinterpret_cast<const float4*>(mine + 8 * (h0 + k) * kPiecePitch);
                    const float4 u = s[0], v = s[1];
                    z[4 * k] = make_float2(u.x, u.y);
                    z[4 * k + 1] = make_float2(u.z, u.w);
                    z[4 * k + 2] = make_float2(v.x, v.y);
                    z[4 * k + 3] = make_float2(v.z, v.w);
                }
                if (p.e.bias) {
#pragma unroll
                    for (int j = 0; j < 4 * H; ++j) z[j] = add2(z[j], b[j & 3]);
                }
                if (p.e.in) {
                    if (!kAhead) {
#pragma unroll
                        for (int k = 0; k < H; ++k) load_one(p, k, r0 + 8 * (h0 + k), col);
                    }
                    const bool second = kAhead && H == 1 && h0;
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        to_pairs<F32, 8>(second ? in[1] : in[k], x, 4 * k);
                        to_pairs<F32, 8>(second ? in2[1] : in2[k], y, 4 * k);
                    }
                }
                const auto store = [&](const float2(&d)[4 * H], const float2(&w)[4 * H]) {
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        const int row = r0 + 8 * (h0 + k);
                        if (row >= p.m) continue;
                        if (p.e.out2) from_pairs<F32, 8>(w, 4 * k).store(p.e.out2, row * p.e.ld_out2 + col);
                        from_pairs<F32, 8>(d, 4 * k).store(p.d, row * p.ldd + col);
                    }
                };
                if constexpr (SHORT) finish_short<F32>(p.e, z, x, y, store);
                else finish_elements<F32>(p.e, z, x, y, store);
            }
        } else {
            const int col = col0 + lane, rows = p.m - row0;
            if (col >= p.n) return;
            constexpr int64_t es = F32 ? 4 : 2;
            const auto at = [&](const void* base, int64_t ld) { return static_cast<const char*>(base) + (row0 * ld + col) * es; };
            float2 z[8], x[8], y[8];
            const auto put = [&](const float2(&v)[8], const void* base, int64_t ld) {
                char* q = const_cast<char*>(at(base, ld));
                const bool whole = rows >= 16;
#pragma unroll
                for (int j = 0; j < 16; ++j, q += ld * es) {
                    const float one[1] = {j & 1 ? v[j / 2].y : v[j / 2].x};
                    if (whole || j < rows) RowVec<F32, 1>::put(q, 0, one);
                }
            };
            const auto pairs = [](const RowVec<F32, 1>(&v)[VEC ? 1 : 16], float2(&to)[8]) {
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float a[1], c[1];
                    v[VEC ? 0 : j].get(a);
                    v[VEC ? 0 : j + 1].get(c);
                    to[j / 2] = make_float2(a[0], c[0]);
                }
            };
            pairs(cin, x);
            pairs(cin2, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[j] = add2(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), b[0]);
            finish_short<F32>(p.e, z, x, y, [&](const float2(&d)[8], const float2(&w)[8]) {
                if (p.e.out2) put(w, p.e.out2, p.e.ld_out2);
                put(d, p.d, p.ldd);
            });
        }
    }
};

}  // namespace hm
