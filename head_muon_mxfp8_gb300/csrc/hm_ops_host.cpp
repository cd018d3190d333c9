// Entry points of the operators around the update: argument checks on the
// host, then one or two launches.  Nothing is launched when a check fails.
#include "hm.h"
#include "hm_internal.h"
#include "hm_ops.h"

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

namespace {

inline hm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HM_OK : HM_ERR_CUDA; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Bytes of [rows][ld] of which the last row ends after `cols` elements.
struct Span {
    uintptr_t lo, hi;
};
Span span(const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0 || cols <= 0) return {a, a};
    return {a, a + static_cast<uintptr_t>(((rows - 1) * ld + cols) * elem)};
}
bool overlap(const Span& x, const Span& y) { return x.lo < y.hi && y.lo < x.hi; }

int64_t tiled_bytes(int64_t rows, int64_t k) { return up(rows, 128) / 128 * (up(k, 128) / 128) * 512; }

bool elem_size(hm_dtype t, int64_t* es) {
    if (t == HM_BF16) *es = 2;
    else if (t == HM_F32) *es = 4;
    else return false;
    return true;
}

constexpr int64_t kMaxDim = INT32_MAX - 256;   // tile coordinates and row counts stay in 32 bits
constexpr int64_t kMaxPitch = int64_t(1) << 40;

// Whether [rows][ld] of `elem` bytes is larger than any address space (2^56 bytes), so
// that offsets and the ends of spans would leave 64 bits.
bool too_far(int64_t rows, int64_t ld, int64_t elem) {
    return rows > 0 && ld > 0 && ld > (int64_t(1) << 56) / elem / rows;
}

}  // namespace

bool hm::inject_mx_timeout() {
    const char* v = std::getenv("HM_INJECT_MX_WAIT_TIMEOUT");
    return v && v[0] == '1';
}

extern "C" hm_status mxfp8_tiled_scale_bytes(int64_t rows, int64_t k, size_t* bytes) {
    if (!bytes || rows < 0 || k < 0) return HM_ERR_ARG;
    if (rows > kMaxDim || k > kMaxDim) return HM_ERR_GEOMETRY;
    if (k % HM_MX_BLOCK) return HM_ERR_ALIGN;
    *bytes = static_cast<size_t>(tiled_bytes(rows, k));
    return HM_OK;
}

namespace {

// The matrices of D's shape that an epilogue reads and writes, in this order: in, in2, out2.
struct EpilogueUse {
    const void* p;
    int64_t ld;
    bool takes, needs;  // of the form
};
void epilogue_use(const hm_epilogue& e, EpilogueUse (&u)[3]) {
    const bool gated = e.form == HM_EPI_GATED_GRADIENT;
    u[0] = {e.in, e.ld_in, true, e.form != HM_EPI_FORWARD};
    u[1] = {e.in2, e.ld_in2, gated, gated};
    u[2] = {e.out2, e.ld_out2, e.form != HM_EPI_GRADIENT, gated};
}

// The checks of both products, the epilogue's too where there is one; *go: something to launch.
hm_status gemm_args(const uint8_t* a, int64_t lda, const uint8_t* a_scales, const uint8_t* b, int64_t ldb,
                    const uint8_t* b_scales, int64_t m, int64_t n, int64_t k, void* d, int64_t ldd, hm_dtype d_dtype,
                    int accumulate, const hm_epilogue* e, hm::MxGemmArgs* p, bool* go) {
    *go = false;
    int64_t es = 0;
    if (m < 0 || n < 0 || k < 0) return HM_ERR_ARG;
    if (!elem_size(d_dtype, &es) || (accumulate && d_dtype != HM_F32)) return HM_ERR_DTYPE;
    EpilogueUse use[3] = {};
    if (e) {
        if (e->form < HM_EPI_FORWARD || e->form > HM_EPI_GATED_GRADIENT || e->activation < HM_ACT_NONE ||
            e->activation > HM_ACT_SILU)
            return HM_ERR_ARG;
        epilogue_use(*e, use);
        if (e->bias && e->form > HM_EPI_GATED) return HM_ERR_ARG;
        for (const EpilogueUse& u : use)
            if (u.p && !u.takes) return HM_ERR_ARG;
    }
    if (m > kMaxDim || n > kMaxDim || k > kMaxDim || lda > kMaxDim || ldb > kMaxDim || ldd > kMaxPitch ||
        too_far(m, lda, 1) || too_far(n, ldb, 1) || too_far(m, ldd, es))
        return HM_ERR_GEOMETRY;
    for (const EpilogueUse& u : use)
        if (u.p && (u.ld > kMaxPitch || too_far(m, u.ld, es))) return HM_ERR_GEOMETRY;
    if (m == 0 || n == 0) return HM_OK;
    if (!d || ldd < n || (k && (!a || !a_scales || !b || !b_scales || lda < k || ldb < k))) return HM_ERR_ARG;
    for (const EpilogueUse& u : use)
        if (u.p ? u.ld < n : u.needs) return HM_ERR_ARG;
    if (k % HM_MX_BLOCK || !aligned(d, es)) return HM_ERR_ALIGN;
    if (k && (lda % 16 || ldb % 16 || !aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 16) ||
              !aligned(b_scales, 16)))
        return HM_ERR_ALIGN;
    if (e && !aligned(e->bias, 4)) return HM_ERR_ALIGN;
    for (const EpilogueUse& u : use)
        if (!aligned(u.p, es)) return HM_ERR_ALIGN;
    const Span outs[2] = {span(d, m, ldd, n, es), span(use[2].p, m, use[2].ld, n, es)};
    for (int i = 0; i < 2; ++i) {
        const Span& out = outs[i];
        if (k && (overlap(out, span(a, m, lda, k, 1)) || overlap(out, span(b, n, ldb, k, 1)) ||
                  overlap(out, span(a_scales, 1, 0, tiled_bytes(m, k), 1)) ||
                  overlap(out, span(b_scales, 1, 0, tiled_bytes(n, k), 1))))
            return HM_ERR_OVERLAP;
        if (e && overlap(out, span(e->bias, 1, 0, n, 4))) return HM_ERR_OVERLAP;
        // an output may be an input of its shape exactly: a thread reads an element before it writes it
        const void* q = i ? use[2].p : d;
        const int64_t ldq = i ? use[2].ld : ldd;
        for (int j = 0; j < 2; ++j)
            if (!(q == use[j].p && ldq == use[j].ld) && overlap(out, span(use[j].p, m, use[j].ld, n, es)))
                return HM_ERR_OVERLAP;
    }
    if (overlap(outs[0], outs[1])) return HM_ERR_OVERLAP;
    if (up(m, 128) / 128 * (up(n, 128) / 128) > INT32_MAX) return HM_ERR_GEOMETRY;
    const hm_status st = hm::check_arch();
    if (st != HM_OK) return st;
    std::memset(p, 0, sizeof(*p));
    p->sa = a_scales;
    p->sb = b_scales;
    p->d = d;
    p->ldd = ldd;
    p->m = static_cast<int32_t>(m);
    p->n = static_cast<int32_t>(n);
    p->k = static_cast<int32_t>(k);
    p->d_f32 = d_dtype == HM_F32;
    p->accumulate = accumulate != 0;
    if (e) {
        p->epilogue = 1;
        p->e = {e->form, e->activation, e->bias, e->in, e->in2, e->out2, e->ld_in, e->ld_in2, e->ld_out2};
    }
    *go = true;
    return HM_OK;
}

}  // namespace

extern "C" hm_status mxfp8_gemm(const uint8_t* a, int64_t lda, const uint8_t* a_scales, const uint8_t* b, int64_t ldb,
                                const uint8_t* b_scales, int64_t m, int64_t n, int64_t k, void* d, int64_t ldd,
                                hm_dtype d_dtype, int accumulate, void* stream) {
    hm::MxGemmArgs p;
    bool go;
    const hm_status st = gemm_args(a, lda, a_scales, b, ldb, b_scales, m, n, k, d, ldd, d_dtype, accumulate, nullptr, &p, &go);
    if (st != HM_OK || !go) return st;
    return cuda_status(hm::launch_mx_gemm(a, lda, b, ldb, p, static_cast<cudaStream_t>(stream)));
}

extern "C" hm_status mxfp8_gemm_epilogue(const uint8_t* a, int64_t lda, const uint8_t* a_scales, const uint8_t* b,
                                         int64_t ldb, const uint8_t* b_scales, int64_t m, int64_t n, int64_t k, void* d,
                                         int64_t ldd, hm_dtype d_dtype, const hm_epilogue* epilogue, void* stream) {
    if (!epilogue) return HM_ERR_ARG;
    hm::MxGemmArgs p;
    bool go;
    const hm_status st = gemm_args(a, lda, a_scales, b, ldb, b_scales, m, n, k, d, ldd, d_dtype, 0, epilogue, &p, &go);
    if (st != HM_OK || !go) return st;
    return cuda_status(hm::launch_mx_gemm(a, lda, b, ldb, p, static_cast<cudaStream_t>(stream)));
}

namespace {

hm_status gemm_form(int64_t m, int64_t n, int64_t k, hm_dtype d_dtype, bool epilogue, int32_t* tile, int32_t* parts,
                    int32_t* sums) {
    int64_t es = 0;
    if (!tile || !parts || !sums || m <= 0 || n <= 0 || k <= 0) return HM_ERR_ARG;
    if (!elem_size(d_dtype, &es)) return HM_ERR_DTYPE;
    if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return HM_ERR_GEOMETRY;
    if (k % HM_MX_BLOCK) return HM_ERR_ALIGN;
    const hm_status st = hm::check_arch();
    if (st != HM_OK) return st;
    hm::MxGemmArgs p;
    std::memset(&p, 0, sizeof(p));
    p.m = static_cast<int32_t>(m);
    p.n = static_cast<int32_t>(n);
    p.k = static_cast<int32_t>(k);
    p.d_f32 = d_dtype == HM_F32;
    p.epilogue = epilogue;
    hm::MxGemmForm f;
    const hm_status ok = cuda_status(hm::mx_gemm_form(p, &f));
    if (ok == HM_OK) *tile = f.tile, *parts = f.parts, *sums = f.sums;
    return ok;
}

}  // namespace

extern "C" hm_status mxfp8_gemm_form(int64_t m, int64_t n, int64_t k, hm_dtype d_dtype, int32_t* tile, int32_t* parts,
                                     int32_t* sums) {
    return gemm_form(m, n, k, d_dtype, false, tile, parts, sums);
}

extern "C" hm_status mxfp8_gemm_epilogue_form(int64_t m, int64_t n, int64_t k, hm_dtype d_dtype, int32_t* tile,
                                              int32_t* parts, int32_t* sums) {
    return gemm_form(m, n, k, d_dtype, true, tile, parts, sums);
}

namespace {

// The checks of both quantizations; *go: something to launch.
hm_status quantize_args(const void* x, hm_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx, const float* row_mul,
                        const float* col_mul, int block, uint8_t* q, int64_t ldq, uint8_t* s, uint8_t* qt, int64_t ldqt,
                        uint8_t* st, const Span (&more)[2], hm::QuantArgs* a, bool* go) {
    *go = false;
    int64_t es = 0;
    if (rows < 0 || cols < 0 || (block != 32 && block != 128)) return HM_ERR_ARG;
    if (!elem_size(x_dtype, &es)) return HM_ERR_DTYPE;
    if ((!q && !qt) || !q != !s || !qt != !st) return HM_ERR_ARG;
    if (rows > (int64_t(1) << 22) || cols > (int64_t(1) << 30) || ldx > kMaxPitch || ldq > kMaxPitch || ldqt > kMaxPitch ||
        too_far(rows, ldx, es) || too_far(rows, ldq, 1) || too_far(cols, ldqt, 1))
        return HM_ERR_GEOMETRY;
    if (rows == 0 || cols == 0) return HM_OK;
    const int64_t cols32 = up(cols, 32), rows32 = up(rows, 32);
    if (!x || ldx < cols || (q && ldq < cols32) || (qt && ldqt < rows32)) return HM_ERR_ARG;
    if (!aligned(x, es) || !aligned(row_mul, 4) || !aligned(col_mul, 4)) return HM_ERR_ALIGN;
    if (q && (ldq % 16 || !aligned(q, 16) || !aligned(s, 16))) return HM_ERR_ALIGN;
    if (qt && (ldqt % 16 || !aligned(qt, 16) || !aligned(st, 16))) return HM_ERR_ALIGN;
    const Span all[] = {span(x, rows, ldx, cols, es),
                        span(row_mul, 1, 0, rows, 4),
                        span(col_mul, 1, 0, cols, 4),
                        span(q, rows, ldq, cols32, 1),
                        span(s, 1, 0, tiled_bytes(rows, cols32), 1),
                        span(qt, cols, ldqt, rows32, 1),
                        span(st, 1, 0, tiled_bytes(cols, rows32), 1)};
    for (int i = 3; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(all[i], all[j])) return HM_ERR_OVERLAP;
    for (const Span& m : more)
        for (const Span& x1 : all)
            if (overlap(m, x1)) return HM_ERR_OVERLAP;
    const hm_status ok = hm::check_arch();
    if (ok != HM_OK) return ok;
    std::memset(a, 0, sizeof(*a));
    a->x = x;
    a->rows = rows;
    a->cols = cols;
    a->ldx = ldx;
    a->row_mul = row_mul;
    a->col_mul = col_mul;
    a->q = q;
    a->ldq = ldq;
    a->s = s;
    a->qt = qt;
    a->ldqt = ldqt;
    a->st = st;
    a->block = block;
    a->vec = aligned(x, 16) && ldx * es % 16 == 0;
    a->col_vec = col_mul && aligned(col_mul, 16);
    *go = true;
    return HM_OK;
}

}  // namespace

extern "C" hm_status mxfp8_quantize(const void* x, hm_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                    const float* row_mul, const float* col_mul, int block, uint8_t* q, int64_t ldq,
                                    uint8_t* s, uint8_t* qt, int64_t ldqt, uint8_t* st, void* stream) {
    hm::QuantArgs a;
    bool go;
    const Span none[2] = {};
    const hm_status ok = quantize_args(x, x_dtype, rows, cols, ldx, row_mul, col_mul, block, q, ldq, s, qt, ldqt, st, none, &a, &go);
    if (ok != HM_OK || !go) return ok;
    return cuda_status(hm::launch_quantize(a, x_dtype == HM_F32, static_cast<cudaStream_t>(stream)));
}

extern "C" hm_status mxfp8_quantize_bias_workspace(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes || rows < 0 || cols < 0) return HM_ERR_ARG;
    if (rows > (int64_t(1) << 22) || cols > (int64_t(1) << 30)) return HM_ERR_GEOMETRY;
    *bytes = rows > 128 ? static_cast<size_t>(up(rows, 128) / 128) * static_cast<size_t>(cols) * 4 : 0;
    return HM_OK;
}

extern "C" hm_status mxfp8_quantize_bias(const void* x, hm_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx, int block,
                                         uint8_t* q, int64_t ldq, uint8_t* s, uint8_t* qt, int64_t ldqt, uint8_t* st,
                                         float* dbias, int accumulate, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    if (rows < 0 || cols < 0) return HM_ERR_ARG;
    if (rows > (int64_t(1) << 22) || cols > (int64_t(1) << 30)) return HM_ERR_GEOMETRY;
    if (cols && !dbias) return HM_ERR_ARG;
    if (!aligned(dbias, 4) || !aligned(workspace, 16)) return HM_ERR_ALIGN;
    size_t need = 0;
    mxfp8_quantize_bias_workspace(rows, cols, &need);
    const Span sums[2] = {span(dbias, 1, 0, cols, 4), span(workspace, 1, 0, static_cast<int64_t>(need), 1)};
    if (overlap(sums[0], sums[1])) return HM_ERR_OVERLAP;
    if (rows && need && (!workspace || workspace_bytes < need)) return HM_ERR_WORKSPACE;
    hm::QuantArgs a;
    bool go;
    hm_status ok = quantize_args(x, x_dtype, rows, cols, ldx, nullptr, nullptr, block, q, ldq, s, qt, ldqt, st, sums, &a, &go);
    if (ok != HM_OK) return ok;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!go) {  // no rows: the empty sum
        if (!cols || accumulate) return HM_OK;
        if ((ok = hm::check_arch()) != HM_OK) return ok;
        return cuda_status(hm::launch_bias_sums(nullptr, 0, cols, 0, dbias, cs));
    }
    a.sums = need ? static_cast<float*>(workspace) : dbias;
    a.sums_add = !need && accumulate;
    ok = cuda_status(hm::launch_quantize(a, x_dtype == HM_F32, cs));
    if (ok != HM_OK || !need) return ok;
    return cuda_status(hm::launch_bias_sums(a.sums, up(rows, 128) / 128, cols, accumulate != 0, dbias, cs));
}


extern "C" hm_status rmsnorm_mxfp8(const void* x, int64_t ldx, const void* res, void* h, int64_t ldh, hm_dtype dtype,
                                   int64_t rows, int64_t d, const float* gamma, float eps, int block, float* rstd,
                                   uint8_t* q, uint8_t* s, void* stream) {
    int64_t es = 0;
    if (rows < 0 || d < 0 || (block != 32 && block != 128) || !(eps >= 0.f)) return HM_ERR_ARG;
    if (!elem_size(dtype, &es)) return HM_ERR_DTYPE;
    if (d > HM_RMSNORM_MAX_D || rows > kMaxDim || ldx > kMaxPitch || ldh > kMaxPitch || too_far(rows, ldx, es) ||
        too_far(rows, ldh, es))
        return HM_ERR_GEOMETRY;
    if (rows == 0 || d == 0) return HM_OK;
    if (!x || !gamma || !rstd || !q || !s || ldx < d || ((res || h) && ldh < d) || (res && !h)) return HM_ERR_ARG;
    if (d % HM_MX_BLOCK || ldx % 8 || ((res || h) && ldh % 8)) return HM_ERR_ALIGN;
    for (const void* p : {x, res, static_cast<const void*>(h), static_cast<const void*>(gamma),
                          static_cast<const void*>(q), static_cast<const void*>(s)})
        if (!aligned(p, 16)) return HM_ERR_ALIGN;
    if (!aligned(rstd, 4)) return HM_ERR_ALIGN;
    // h may be x or res itself (a row is read before it is written), nothing else may overlap an output
    const Span in[] = {span(x, rows, ldx, d, es), span(res, rows, ldh, d, es), span(gamma, 1, 0, d, 4)};
    const Span out[] = {span(h, rows, ldh, d, es), span(rstd, 1, 0, rows, 4), span(q, 1, 0, rows * d, 1),
                        span(s, 1, 0, tiled_bytes(rows, d), 1)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j) {
            const bool same = i == 0 && ((j == 0 && h == x && ldh == ldx) || (j == 1 && h == res));
            if (!same && overlap(out[i], in[j])) return HM_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return HM_ERR_OVERLAP;
    }
    const hm_status st = hm::check_arch();
    if (st != HM_OK) return st;
    hm::RmsArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.res = res;
    a.h = h;
    a.ldx = ldx;
    a.ldh = ldh;
    a.rows = rows;
    a.d = static_cast<int32_t>(d);
    a.block = block;
    a.gamma = gamma;
    a.eps = eps;
    a.rstd = rstd;
    a.q = q;
    a.s = s;
    return cuda_status(hm::launch_rmsnorm(a, dtype == HM_F32, static_cast<cudaStream_t>(stream)));
}

extern "C" hm_status rmsnorm_backward_workspace(int64_t rows, int64_t d, size_t* bytes) {
    if (!bytes || rows < 0 || d < 0) return HM_ERR_ARG;
    if (d > HM_RMSNORM_MAX_D || rows > kMaxDim) return HM_ERR_GEOMETRY;
    if (d % HM_MX_BLOCK) return HM_ERR_ALIGN;
    *bytes = static_cast<size_t>(hm::rmsnorm_grad_parts(rows, d)) * static_cast<size_t>(d) * 4;
    return HM_OK;
}

extern "C" hm_status rmsnorm_backward(const void* dy, int64_t lddy, const void* dres, const void* h, void* dx,
                                      int64_t ldh, hm_dtype dtype, int64_t rows, int64_t d, const float* gamma,
                                      const float* rstd, float* dgamma, int accumulate, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    int64_t es = 0;
    if (rows < 0 || d < 0) return HM_ERR_ARG;
    if (!elem_size(dtype, &es)) return HM_ERR_DTYPE;
    if (d > HM_RMSNORM_MAX_D || rows > kMaxDim || lddy > kMaxPitch || ldh > kMaxPitch || too_far(rows, lddy, es) ||
        too_far(rows, ldh, es))
        return HM_ERR_GEOMETRY;
    if (d == 0) return HM_OK;
    if (!dgamma) return HM_ERR_ARG;
    if (rows && (!dy || !h || !dx || !gamma || !rstd || lddy < d || ldh < d)) return HM_ERR_ARG;
    if (d % HM_MX_BLOCK || !aligned(dgamma, 4)) return HM_ERR_ALIGN;
    if (rows) {
        if (lddy % 8 || ldh % 8 || !aligned(rstd, 4)) return HM_ERR_ALIGN;
        for (const void* p : {dy, dres, h, static_cast<const void*>(dx), static_cast<const void*>(gamma),
                              static_cast<const void*>(workspace)})
            if (!aligned(p, 16)) return HM_ERR_ALIGN;
        const Span out = span(dx, rows, ldh, d, es), dg = span(dgamma, 1, 0, d, 4);
        const Span ws = span(workspace, 1, 0, static_cast<int64_t>(workspace_bytes), 1);
        const Span in[] = {span(dy, rows, lddy, d, es), span(dres, rows, ldh, d, es), span(h, rows, ldh, d, es),
                           span(gamma, 1, 0, d, 4), span(rstd, 1, 0, rows, 4)};
        for (int j = 0; j < 5; ++j) {
            const bool same = (j == 0 && dx == dy && ldh == lddy) || (j == 1 && dx == dres) || (j == 2 && dx == h);
            if ((!same && overlap(out, in[j])) || overlap(dg, in[j]) || overlap(ws, in[j])) return HM_ERR_OVERLAP;
        }
        if (overlap(out, dg) || overlap(ws, out) || overlap(ws, dg)) return HM_ERR_OVERLAP;
    }
    const hm_status st = hm::check_arch();
    if (st != HM_OK) return st;
    const size_t need = static_cast<size_t>(hm::rmsnorm_grad_parts(rows, d)) * static_cast<size_t>(d) * 4;
    if (need && (!workspace || workspace_bytes < need)) return HM_ERR_WORKSPACE;
    if (!rows && accumulate) return HM_OK;
    hm::RmsGradArgs a;
    std::memset(&a, 0, sizeof(a));
    a.dy = dy;
    a.dres = dres;
    a.h = h;
    a.dx = dx;
    a.lddy = lddy;
    a.ldh = ldh;
    a.rows = rows;
    a.d = static_cast<int32_t>(d);
    a.accumulate = accumulate != 0;
    a.gamma = gamma;
    a.rstd = rstd;
    a.dgamma = dgamma;
    a.partials = static_cast<float*>(workspace);
    return cuda_status(hm::launch_rmsnorm_grad(a, dtype == HM_F32, static_cast<cudaStream_t>(stream)));
}

namespace {

// [rows][heads] of head_dim elements, in bytes: the outer of the two strides, how far
// the rest reaches from one outer step, and the whole span.
struct Block3 {
    Span all;
    int64_t pitch, width;  // pitch 0: one outer step
};
Block3 block3(const void* p, int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t dim, int64_t es) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const bool row_outer = heads == 1 || (rows > 1 && row >= head);
    const int64_t n_out = row_outer ? rows : heads, out = row_outer ? row : head;
    const int64_t n_in = row_outer ? heads : rows, in = row_outer ? head : row;
    Block3 b;
    b.width = ((n_in - 1) * in + dim) * es;
    b.pitch = n_out > 1 ? out * es : 0;
    b.all = {a, p ? a + static_cast<uintptr_t>((n_out - 1) * out * es + b.width) : a};
    return b;
}
// Blocks with one pitch may interleave (queries and keys of a packed projection);
// otherwise the spans decide.
bool overlap(const Block3& x, const Block3& y) {
    if (!overlap(x.all, y.all)) return false;
    const int64_t pitch = x.pitch ? x.pitch : y.pitch;
    if (!pitch || (x.pitch && y.pitch && x.pitch != y.pitch) || x.width > pitch || y.width > pitch) return true;
    const int64_t d = static_cast<int64_t>((y.all.lo - x.all.lo) % static_cast<uintptr_t>(pitch));
    const int64_t at = y.all.lo >= x.all.lo ? d : (pitch - static_cast<int64_t>((x.all.lo - y.all.lo) % static_cast<uintptr_t>(pitch))) % pitch;
    return at < x.width || at + y.width > pitch;
}

// One strided array of a group: its pointer and strides.
struct HeadMatrix {
    const void* p;
    int64_t row, head;
};
constexpr int64_t kMaxHeads = 65536;

// No address twice: heads inside a row, or rows inside a head.
bool apart(const HeadMatrix& m, int64_t rows, int64_t heads, int64_t dim) {
    if (rows > 1 && heads > 1)
        return (m.head >= dim && m.row >= (heads - 1) * m.head + dim) || (m.row >= dim && m.head >= (rows - 1) * m.row + dim);
    return (rows == 1 || m.row >= dim) && (heads == 1 || m.head >= dim);
}
bool same(const HeadMatrix& x, const HeadMatrix& y) { return x.p == y.p && x.row == y.row && x.head == y.head; }

hm_status head_matrix(const HeadMatrix& m, int64_t rows, int64_t heads, int64_t dim, int64_t es, bool output) {
    if (!m.p || m.row < 0 || m.head < 0) return HM_ERR_ARG;
    if (m.row > kMaxPitch || m.head > kMaxPitch || too_far(rows, m.row, es) || too_far(heads, m.head, es)) return HM_ERR_GEOMETRY;
    if (!aligned(m.p, es)) return HM_ERR_ALIGN;
    return output && !apart(m, rows, heads, dim) ? HM_ERR_ARG : HM_OK;
}

// A call's groups, all of them.
struct HeadCall {
    hm::HeadGroup g[HM_HEAD_GROUPS];
    int n;
};
// Launches them by pairs, whose groups share the CTAs.
template <class Launch>
hm_status by_pairs(hm::HeadArgs& a, const HeadCall& call, const Launch& launch) {
    static_assert(hm::kHeadGroups == 2, "pairs");
    for (int i = 0; i < call.n; i += 2) {
        a.n = std::min(2, call.n - i);
        std::memset(a.g, 0, sizeof(a.g));
        a.all_heads = a.all_groups = 0;
        for (int k = 0; k < a.n; ++k) {
            a.g[k] = call.g[i + k];
            a.all_heads += a.g[k].heads;
            a.all_groups += a.g[k].heads > 0;
        }
        const hm_status ok = cuda_status(launch(a));
        if (ok != HM_OK) return ok;
    }
    return HM_OK;
}

// What both calls check of their common arguments, and a's part of them.
hm_status head_common(int n_groups, hm_dtype dtype, int64_t rows, int64_t head_dim, float eps, const hm_rotation* rot,
                      int64_t* es, hm::HeadArgs* a) {
    if (n_groups < 0 || rows < 0 || head_dim < 0 || !(eps >= 0.f)) return HM_ERR_ARG;
    if (!elem_size(dtype, es)) return HM_ERR_DTYPE;
    if (n_groups > HM_HEAD_GROUPS || rows > kMaxDim || head_dim > HM_HEAD_MAX_DIM || head_dim % 2) return HM_ERR_GEOMETRY;
    std::memset(a, 0, sizeof(*a));
    a->rows = rows;
    a->dim = static_cast<int32_t>(head_dim);
    a->eps = eps;
    if (rot && rot->rot_dim) {
        if (rot->rot_dim < 0 || (rot->layout != HM_ROPE_HALF && rot->layout != HM_ROPE_PAIRS) || !std::isfinite(rot->scale))
            return HM_ERR_ARG;
        if (rot->rot_dim > head_dim || rot->rot_dim % 2) return HM_ERR_GEOMETRY;
        if (rows && (!rot->turns || !rot->positions)) return HM_ERR_ARG;
        if (!aligned(rot->turns, 8) || !aligned(rot->positions, 8)) return HM_ERR_ALIGN;
        a->turns = rot->turns;
        a->positions = rot->positions;
        a->rot = rot->rot_dim;
        a->pairs = rot->layout == HM_ROPE_PAIRS;
        a->scale = rot->scale;
    }
    return HM_OK;
}

// What a call reads besides its matrices.
void head_small(const hm::HeadArgs& a, Span (&s)[2]) {
    s[0] = span(a.turns, 1, 0, a.rot / 2, 8);
    s[1] = span(a.positions, 1, 0, a.rows, 8);
}

}  // namespace

extern "C" hm_status head_norm_rope(const hm_head_group* groups, int n_groups, hm_dtype dtype, int64_t rows,
                                    int64_t head_dim, float eps, const hm_rotation* rotation, void* stream) {
    int64_t es = 0;
    hm::HeadArgs a;
    HeadCall call = {};
    hm_status ok = head_common(n_groups, dtype, rows, head_dim, eps, rotation, &es, &a);
    if (ok != HM_OK) return ok;
    if (n_groups && !groups) return HM_ERR_ARG;
    Span small[2];
    head_small(a, small);
    Block3 x[HM_HEAD_GROUPS], y[HM_HEAD_GROUPS];
    call.n = 0;
    for (int i = 0; i < n_groups; ++i) {
        const hm_head_group& g = groups[i];
        if (g.heads < 0) return HM_ERR_ARG;
        if (g.heads > kMaxHeads) return HM_ERR_GEOMETRY;
        if (!aligned(g.gamma, 4)) return HM_ERR_ALIGN;
        if (!g.heads || !rows || !head_dim) continue;
        const HeadMatrix in = {g.x, g.x_row, g.x_head}, out = {g.y, g.y_row, g.y_head};
        if ((ok = head_matrix(in, rows, g.heads, head_dim, es, false)) != HM_OK) return ok;
        if ((ok = head_matrix(out, rows, g.heads, head_dim, es, true)) != HM_OK) return ok;
        x[call.n] = block3(g.x, rows, g.x_row, g.heads, g.x_head, head_dim, es);
        y[call.n] = block3(g.y, rows, g.y_row, g.heads, g.y_head, head_dim, es);
        hm::HeadGroup& to = call.g[call.n++];
        to.in = g.x;
        to.in_row = g.x_row;
        to.in_head = g.x_head;
        to.out = g.y;
        to.out_row = g.y_row;
        to.out_head = g.y_head;
        to.gamma = g.gamma;
        to.heads = g.heads;
    }
    for (int i = 0; i < call.n; ++i) {
        for (int j = 0; j < call.n; ++j) {
            const bool in_place = i == j && same({call.g[i].in, call.g[i].in_row, call.g[i].in_head}, {call.g[i].out, call.g[i].out_row, call.g[i].out_head});
            if ((!in_place && overlap(y[i], x[j])) || (j < i && overlap(y[i], y[j])) ||
                overlap(y[i].all, span(call.g[j].gamma, 1, 0, head_dim, 4)))
                return HM_ERR_OVERLAP;
        }
        if (overlap(y[i].all, small[0]) || overlap(y[i].all, small[1])) return HM_ERR_OVERLAP;
    }
    if (!call.n) return HM_OK;
    if ((ok = hm::check_arch()) != HM_OK) return ok;
    return by_pairs(a, call, [&](hm::HeadArgs& pair) {
        pair.width = hm::head_width(pair, es);
        return hm::launch_heads(pair, dtype == HM_F32, static_cast<cudaStream_t>(stream));
    });
}

namespace {

// Whether a gradient call has anything to do for a group.
bool takes_part(const hm_head_grad& g, int64_t rows) { return (g.heads && rows) || g.dgamma; }

// Floats of dgamma's partial sums of group i: a row per CTA, which its launch deals out to the
// pair that it takes (by_pairs, of the groups that take part).
size_t grad_partials(const hm_head_grad* groups, int n, int i, int64_t rows, int64_t head_dim) {
    const hm_head_grad& g = groups[i];
    if (!g.dgamma || !g.heads || !rows) return 0;
    int before = 0;
    for (int k = 0; k < i; ++k) before += takes_part(groups[k], rows);
    int heads = 0, live = 0, place = 0;
    for (int k = 0; k < n; ++k) {
        if (!takes_part(groups[k], rows)) continue;
        if (place++ / 2 != before / 2) continue;
        heads += groups[k].heads;
        live += groups[k].heads > 0;
    }
    return static_cast<size_t>(hm::head_grad_parts(rows, g.heads, heads, live)) * static_cast<size_t>(head_dim);
}

}  // namespace

extern "C" hm_status head_norm_rope_backward_workspace(const hm_head_grad* groups, int n_groups, int64_t rows,
                                                       int64_t head_dim, size_t* bytes) {
    if (!bytes || n_groups < 0 || rows < 0 || head_dim < 0 || (n_groups && !groups)) return HM_ERR_ARG;
    if (n_groups > HM_HEAD_GROUPS || rows > kMaxDim || head_dim > HM_HEAD_MAX_DIM || head_dim % 2) return HM_ERR_GEOMETRY;
    for (int i = 0; i < n_groups; ++i) {
        if (groups[i].heads < 0) return HM_ERR_ARG;
        if (groups[i].heads > kMaxHeads) return HM_ERR_GEOMETRY;
    }
    size_t floats = 0;
    for (int i = 0; i < n_groups; ++i) floats += grad_partials(groups, n_groups, i, rows, head_dim);
    *bytes = floats * 4;
    return HM_OK;
}

extern "C" hm_status head_norm_rope_backward(const hm_head_grad* groups, int n_groups, hm_dtype dtype, int64_t rows,
                                             int64_t head_dim, float eps, const hm_rotation* rotation, void* workspace,
                                             size_t workspace_bytes, void* stream) {
    int64_t es = 0;
    hm::HeadArgs a;
    HeadCall call = {};
    hm_status ok = head_common(n_groups, dtype, rows, head_dim, eps, rotation, &es, &a);
    if (ok != HM_OK) return ok;
    if (n_groups && !groups) return HM_ERR_ARG;
    if (!aligned(workspace, 16)) return HM_ERR_ALIGN;
    Span small[3];
    Span rot[2];
    head_small(a, rot);
    small[0] = rot[0];
    small[1] = rot[1];
    small[2] = span(workspace, 1, 0, static_cast<int64_t>(workspace_bytes), 1);
    Block3 dy[HM_HEAD_GROUPS], x[HM_HEAD_GROUPS], dx[HM_HEAD_GROUPS];
    Span dg[HM_HEAD_GROUPS];
    int from[HM_HEAD_GROUPS];
    call.n = 0;
    for (int i = 0; i < n_groups; ++i) {
        const hm_head_grad& g = groups[i];
        if (g.heads < 0 || (g.dgamma && !g.gamma)) return HM_ERR_ARG;
        if (g.heads > kMaxHeads) return HM_ERR_GEOMETRY;
        if (!aligned(g.gamma, 4) || !aligned(g.dgamma, 4)) return HM_ERR_ALIGN;
        if (!head_dim) continue;
        const bool live = g.heads && rows;
        if (!takes_part(g, rows)) continue;
        const int k = call.n++;
        from[k] = i;
        hm::HeadGroup& to = call.g[k];
        dg[k] = span(g.dgamma, 1, 0, head_dim, 4);
        to.gamma = g.gamma;
        to.dgamma = g.dgamma;
        to.accumulate = g.accumulate != 0;
        dy[k] = x[k] = dx[k] = Block3{{0, 0}, 0, 0};
        if (!live) continue;
        const HeadMatrix in = {g.dy, g.dy_row, g.dy_head}, xx = {g.x, g.x_row, g.x_head}, out = {g.dx, g.dx_row, g.dx_head};
        if ((ok = head_matrix(in, rows, g.heads, head_dim, es, false)) != HM_OK) return ok;
        if (g.gamma && (ok = head_matrix(xx, rows, g.heads, head_dim, es, false)) != HM_OK) return ok;
        if ((ok = head_matrix(out, rows, g.heads, head_dim, es, true)) != HM_OK) return ok;
        dy[k] = block3(g.dy, rows, g.dy_row, g.heads, g.dy_head, head_dim, es);
        if (g.gamma) x[k] = block3(g.x, rows, g.x_row, g.heads, g.x_head, head_dim, es);
        dx[k] = block3(g.dx, rows, g.dx_row, g.heads, g.dx_head, head_dim, es);
        to.in = g.dy;
        to.in_row = g.dy_row;
        to.in_head = g.dy_head;
        if (g.gamma) {
            to.x = g.x;
            to.x_row = g.x_row;
            to.x_head = g.x_head;
        }
        to.out = g.dx;
        to.out_row = g.dx_row;
        to.out_head = g.dx_head;
        to.heads = g.heads;
    }
    for (int i = 0; i < call.n; ++i) {
        const HeadMatrix out = {call.g[i].out, call.g[i].out_row, call.g[i].out_head};
        for (int j = 0; j < call.n; ++j) {
            const Span gamma = span(call.g[j].gamma, 1, 0, head_dim, 4);
            const bool is_dy = i == j && same(out, {call.g[i].in, call.g[i].in_row, call.g[i].in_head});
            const bool is_x = i == j && same(out, {call.g[i].x, call.g[i].x_row, call.g[i].x_head});
            if ((!is_dy && overlap(dx[i], dy[j])) || (!is_x && overlap(dx[i], x[j])) || (j < i && overlap(dx[i], dx[j])) ||
                overlap(dx[i].all, gamma) || overlap(dx[i].all, dg[j]) || overlap(dg[i], dy[j].all) || overlap(dg[i], x[j].all) ||
                overlap(dg[i], gamma) || (j < i && overlap(dg[i], dg[j])))
                return HM_ERR_OVERLAP;
        }
        for (int j = 0; j < 3; ++j)
            if (overlap(dx[i].all, small[j]) || overlap(dg[i], small[j])) return HM_ERR_OVERLAP;
        if (overlap(small[2], dy[i].all) || overlap(small[2], x[i].all) || overlap(small[2], span(call.g[i].gamma, 1, 0, head_dim, 4)))
            return HM_ERR_OVERLAP;
    }
    if (overlap(small[2], small[0]) || overlap(small[2], small[1])) return HM_ERR_OVERLAP;
    if (!call.n) return HM_OK;
    if ((ok = hm::check_arch()) != HM_OK) return ok;
    size_t floats = 0;
    for (int k = 0; k < call.n; ++k) {
        const size_t part = grad_partials(groups, n_groups, from[k], rows, head_dim);
        if (part) call.g[k].partials = static_cast<float*>(workspace) + floats;
        floats += part;
    }
    if (floats && (!workspace || workspace_bytes < floats * 4)) return HM_ERR_WORKSPACE;
    return by_pairs(a, call, [&](hm::HeadArgs& pair) {
        pair.width = hm::head_width(pair, es);
        return hm::launch_heads_grad(pair, dtype == HM_F32, static_cast<cudaStream_t>(stream));
    });
}

extern "C" hm_status rope_turns(int32_t rot_dim, double theta, int32_t scaling, double factor, double trained,
                                double beta_fast, double beta_slow, uint64_t* turns, float* scale) {
    const double turn = 6.283185307179586476925;  // radians
    if (!turns || !scale || !(theta > 1.0) || !std::isfinite(theta) || scaling < HM_ROPE_UNSCALED || scaling > HM_ROPE_YARN)
        return HM_ERR_ARG;
    if (rot_dim < 2 || rot_dim > HM_HEAD_MAX_DIM || rot_dim % 2) return HM_ERR_GEOMETRY;
    if (scaling == HM_ROPE_UNSCALED) factor = 1.0;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return HM_ERR_ARG;
    double low = 0.0, high = 0.0;
    if (scaling == HM_ROPE_BASE) {
        if (rot_dim == 2) return HM_ERR_GEOMETRY;
        theta *= std::pow(factor, rot_dim / (rot_dim - 2.0));
        if (!std::isfinite(theta)) return HM_ERR_ARG;
    }
    if (scaling == HM_ROPE_YARN) {
        if (!(trained >= 1.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(trained) || !std::isfinite(beta_fast))
            return HM_ERR_ARG;
        // the pair that turns `beta` times over the trained positions
        const auto pair_of = [&](double beta) { return rot_dim * std::log(trained / (beta * turn)) / (2.0 * std::log(theta)); };
        low = std::max(0.0, std::floor(pair_of(beta_fast)));
        high = std::min(rot_dim - 1.0, std::ceil(pair_of(beta_slow)));
        if (!(high > low)) high = low + 0.001;  // no ramp left: a step
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == HM_ROPE_LINEAR) f /= factor;
        if (scaling == HM_ROPE_YARN) {
            const double ramp = std::min(1.0, std::max(0.0, (i - low) / (high - low)));
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        turns[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f / turn, 64)));  // f <= 1: below 2^62
    }
    *scale = scaling == HM_ROPE_YARN ? static_cast<float>(1.0 + 0.1 * std::log(factor)) : 1.f;
    return HM_OK;
}

namespace {

// Appends a tensor to a launch's table; returns the chunks with it.
int64_t add_tensor(hm::ClipHead& h, hm::ClipTensor* table, const hm_grad_tensor& x, int64_t chunks, int vecs) {
    hm::ClipTensor& t = table[h.n++];
    t.src = x.src;
    t.dst = x.dst;
    t.n = x.n;
    t.first = static_cast<int32_t>(chunks);
    t.f32 = x.dtype == HM_F32;
    return chunks + hm::clip_chunks(x.src, x.n, t.f32, vecs);
}

// Checks the list and counts its non-empty tensors and the partial sums of all launches.
hm_status clip_layout(const hm_grad_tensor* t, int n, int64_t* live, int64_t* parts) {
    *live = *parts = 0;
    if (n < 0 || (n > 0 && !t)) return HM_ERR_ARG;
    int64_t chunks = 0, in_launch = 0;
    for (int i = 0; i < n; ++i) {
        int64_t es = 0;
        if (!elem_size(static_cast<hm_dtype>(t[i].dtype), &es)) return HM_ERR_DTYPE;
        if (t[i].n < 0 || (t[i].n > 0 && !t[i].src)) return HM_ERR_ARG;
        if (t[i].n > (int64_t(1) << 42)) return HM_ERR_GEOMETRY;
        if (t[i].n == 0) continue;
        if (!aligned(t[i].src, es) || !aligned(t[i].dst, es)) return HM_ERR_ALIGN;
        const Span src = span(t[i].src, 1, 0, t[i].n, es), dst = span(t[i].dst, 1, 0, t[i].n, es);
        if (t[i].dst && t[i].dst != t[i].src && overlap(src, dst)) return HM_ERR_OVERLAP;
        if (in_launch == hm::kClipTensors) {
            *parts += hm::clip_parts(static_cast<int>(chunks));
            chunks = in_launch = 0;
        }
        chunks += hm::clip_chunks(t[i].src, t[i].n, es == 4, hm::kClipChunkVecs);
        if (chunks > INT32_MAX) return HM_ERR_GEOMETRY;
        ++in_launch;
        ++*live;
    }
    if (in_launch) *parts += hm::clip_parts(static_cast<int>(chunks));
    return HM_OK;
}

}  // namespace

extern "C" hm_status grad_norm_clip_workspace(const hm_grad_tensor* tensors, int n, size_t* bytes) {
    if (!bytes) return HM_ERR_ARG;
    int64_t live = 0, parts = 0;
    const hm_status st = clip_layout(tensors, n, &live, &parts);
    if (st != HM_OK) return st;
    *bytes = static_cast<size_t>(parts) * sizeof(double);
    return HM_OK;
}

extern "C" hm_status grad_norm_clip(const hm_grad_tensor* tensors, int n, float max_norm, float eps, float* stats,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    if (!stats || !(max_norm > 0.f) || !(eps >= 0.f)) return HM_ERR_ARG;
    if (!aligned(stats, 4) || !aligned(workspace, 16)) return HM_ERR_ALIGN;
    int64_t live = 0, parts = 0;
    hm_status ok = clip_layout(tensors, n, &live, &parts);
    if (ok != HM_OK) return ok;
    if (parts > INT32_MAX) return HM_ERR_GEOMETRY;
    if (parts && (!workspace || workspace_bytes < parts * sizeof(double))) return HM_ERR_WORKSPACE;
    // the scaling reads the sums while it writes the tensors and stats
    const Span sums = span(workspace, 1, 0, parts * static_cast<int64_t>(sizeof(double)), 1), result = span(stats, 1, 0, 8, 1);
    if (overlap(sums, result)) return HM_ERR_OVERLAP;
    for (int i = 0; i < n; ++i) {
        const int64_t bytes = tensors[i].n * (tensors[i].dtype == HM_F32 ? 4 : 2);
        const Span src = span(tensors[i].src, 1, 0, bytes, 1), dst = span(tensors[i].dst, 1, 0, bytes, 1);
        if (overlap(sums, src) || overlap(sums, dst) || overlap(result, src) || overlap(result, dst)) return HM_ERR_OVERLAP;
    }
    if ((ok = hm::check_arch()) != HM_OK) return ok;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    hm::ClipHead head;
    std::memset(&head, 0, sizeof(head));
    head.parts = static_cast<int32_t>(parts);
    head.max_norm = max_norm;
    head.eps = eps;
    head.stats = stats;
    head.partials = static_cast<double*>(workspace);
    if (live <= hm::kClipFew) {
        // little data: one launch
        hm::ClipArgs<hm::kClipFew> a;
        a.h = head;
        int64_t chunks = 0;
        for (int i = 0; i < n && chunks <= hm::kClipFewChunks; ++i)
            if (tensors[i].n) chunks = add_tensor(a.h, a.t, tensors[i], chunks, hm::kClipFewChunkVecs);
        a.h.chunks = static_cast<int32_t>(chunks);
        if (chunks <= hm::kClipFewChunks) return cuda_status(hm::launch_clip_few(a, st));
    }
    // two passes over the groups of kClipTensors: every norm launch before the first scaling
    for (int pass = 0; pass < 2; ++pass) {
        int i = 0, part0 = 0;
        do {
            hm::ClipArgs<hm::kClipTensors> a;
            a.h = head;
            int64_t chunks = 0;
            for (; i < n && a.h.n < hm::kClipTensors; ++i)
                if (tensors[i].n) chunks = add_tensor(a.h, a.t, tensors[i], chunks, hm::kClipChunkVecs);
            if (!chunks) break;  // only empty tensors were left
            a.h.chunks = static_cast<int32_t>(chunks);
            a.h.part0 = part0;
            if ((pass == 0 ? hm::launch_clip_norm(a, st) : hm::launch_clip_scale(a, st)) != cudaSuccess) return HM_ERR_CUDA;
            part0 += hm::clip_parts(a.h.chunks);
        } while (i < n);
    }
    return HM_OK;
}
