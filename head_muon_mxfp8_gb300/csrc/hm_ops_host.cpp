// Entry points of the operators around the update: argument checks on the
// host, then one or two launches.  Nothing is launched when a check fails.
#include "hm.h"
#include "hm_internal.h"
#include "hm_ops.h"

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

extern "C" hm_status mxfp8_gemm(const uint8_t* a, int64_t lda, const uint8_t* a_scales, const uint8_t* b, int64_t ldb,
                                const uint8_t* b_scales, int64_t m, int64_t n, int64_t k, void* d, int64_t ldd,
                                hm_dtype d_dtype, int accumulate, void* stream) {
    int64_t es = 0;
    if (m < 0 || n < 0 || k < 0) return HM_ERR_ARG;
    if (!elem_size(d_dtype, &es) || (accumulate && d_dtype != HM_F32)) return HM_ERR_DTYPE;
    if (m > kMaxDim || n > kMaxDim || k > kMaxDim || lda > kMaxDim || ldb > kMaxDim || ldd > kMaxPitch ||
        too_far(m, lda, 1) || too_far(n, ldb, 1) || too_far(m, ldd, es))
        return HM_ERR_GEOMETRY;
    if (m == 0 || n == 0) return HM_OK;
    if (!d || ldd < n || (k && (!a || !a_scales || !b || !b_scales || lda < k || ldb < k))) return HM_ERR_ARG;
    if (k % HM_MX_BLOCK || !aligned(d, es)) return HM_ERR_ALIGN;
    if (k && (lda % 16 || ldb % 16 || !aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 16) ||
              !aligned(b_scales, 16)))
        return HM_ERR_ALIGN;
    if (k) {
        const Span out = span(d, m, ldd, n, es);
        if (overlap(out, span(a, m, lda, k, 1)) || overlap(out, span(b, n, ldb, k, 1)) ||
            overlap(out, span(a_scales, 1, 0, tiled_bytes(m, k), 1)) ||
            overlap(out, span(b_scales, 1, 0, tiled_bytes(n, k), 1)))
            return HM_ERR_OVERLAP;
    }
    if (up(m, 128) / 128 * (up(n, 128) / 128) > INT32_MAX) return HM_ERR_GEOMETRY;
    const hm_status st = hm::check_arch();
    if (st != HM_OK) return st;
    hm::MxGemmArgs p;
    std::memset(&p, 0, sizeof(p));
    p.sa = a_scales;
    p.sb = b_scales;
    p.d = d;
    p.ldd = ldd;
    p.m = static_cast<int32_t>(m);
    p.n = static_cast<int32_t>(n);
    p.k = static_cast<int32_t>(k);
    p.d_f32 = d_dtype == HM_F32;
    p.accumulate = accumulate != 0;
    return cuda_status(hm::launch_mx_gemm(a, lda, b, ldb, p, static_cast<cudaStream_t>(stream)));
}

extern "C" hm_status mxfp8_gemm_form(int64_t m, int64_t n, int64_t k, hm_dtype d_dtype, int32_t* tile, int32_t* parts,
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
    hm::MxGemmForm f;
    const hm_status ok = cuda_status(hm::mx_gemm_form(p, &f));
    if (ok == HM_OK) *tile = f.tile, *parts = f.parts, *sums = f.sums;
    return ok;
}

extern "C" hm_status mxfp8_quantize(const void* x, hm_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                    const float* row_mul, const float* col_mul, int block, uint8_t* q, int64_t ldq,
                                    uint8_t* s, uint8_t* qt, int64_t ldqt, uint8_t* st, void* stream) {
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
    const hm_status ok = hm::check_arch();
    if (ok != HM_OK) return ok;
    hm::QuantArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.row_mul = row_mul;
    a.col_mul = col_mul;
    a.q = q;
    a.ldq = ldq;
    a.s = s;
    a.qt = qt;
    a.ldqt = ldqt;
    a.st = st;
    a.block = block;
    a.vec = aligned(x, 16) && ldx * es % 16 == 0;
    a.col_vec = col_mul && aligned(col_mul, 16);
    return cuda_status(hm::launch_quantize(a, x_dtype == HM_F32, static_cast<cudaStream_t>(stream)));
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
