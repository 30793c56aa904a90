// C entry points of the operators around the mixer: argument checks, workspace sizes and
// dispatch.  See include/ssm_scan.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "layer.h"

namespace ssm {
int abi_fail(int code, const char *msg);
void abi_ok();
void abi_profile_begin(cudaStream_t st);
void abi_profile_end();
}  // namespace ssm

namespace {

using ssm::LaArgs;
using ssm::LaWalk;

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return ssm::abi_fail(code, buf);
}

int need(const void *ptr, const char *name, size_t align) {
    if (!ptr) return fail(SSM_ERR_ARG, "%s is NULL", name);
    if ((uintptr_t)ptr % align) return fail(SSM_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
    return SSM_OK;
}
int may(const void *ptr, const char *name, size_t align) {
    return ptr ? need(ptr, name, align) : SSM_OK;
}

// launch result of `fn` as a status
template <typename F>
int launched(const char *where, void *stream, F fn) {
    cudaStream_t st = (cudaStream_t)stream;
    ssm::abi_profile_begin(st);
    const cudaError_t e = fn(st);
    ssm::abi_profile_end();
    if (e != cudaSuccess) return fail(SSM_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
    ssm::abi_ok();
    return SSM_OK;
}

int check_dtype(int32_t t) {
    return t == SSM_F32 || t == SSM_BF16 ? SSM_OK : fail(SSM_ERR_ARG, "unknown dtype_io %d", t);
}
size_t esize(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

// the stride of a tensor that is read may be 0 (broadcast), that of one that is written not
int check_stride(const char *name, int64_t stride, int64_t extent, int64_t inner, bool written) {
    if (stride < 0) return fail(SSM_ERR_ARG, "%s: negative stride", name);
    if (written && extent > 1 && stride < inner)
        return fail(SSM_ERR_ARG, "%s: stride %lld overlaps rows of %lld values", name,
                    (long long)stride, (long long)inner);
    return SSM_OK;
}
int check_strides3(const char *name, const int64_t *s, const int64_t *extent, int64_t inner,
                   bool written) {
    int order[3], n = 0;   // the dimensions with more than one entry, the smallest stride first
    for (int i = 0; i < 3; ++i) {
        const int rc = check_stride(name, s[i], extent[i], inner, written);
        if (rc) return rc;
        if (extent[i] < 2) continue;
        int j = n++;
        for (; j > 0 && s[order[j - 1]] > s[i]; --j) order[j] = order[j - 1];
        order[j] = i;
    }
    // what is written is nested: each dimension steps over all that the smaller ones span
    double span = (double)inner;
    for (int j = 0; written && j < n; ++j) {
        if ((double)s[order[j]] < span)
            return fail(SSM_ERR_ARG, "%s: stride %lld overlaps other rows", name, (long long)s[order[j]]);
        span += (double)s[order[j]] * (double)(extent[order[j]] - 1);
    }
    return SSM_OK;
}

// A strided tensor of the call, for the checks that an output lies over nothing that other blocks
// read.  `extent` rows of `inner` dense values.
struct Span {
    const char *name;
    const void *p;
    const int64_t *stride, *extent;
    int64_t inner;
    size_t es;
};
// Whether some of n_i s_i (|n_i| bounded by the two extents) and an offset within the rows come to d.
// The dimensions in `order` have falling strides, each over all that the later ones span.
bool meets(const Span &a, const Span &b, const int64_t *st, const int *order, int n, int64_t d) {
    if (n == 0) return d < a.inner && d > -b.inner;
    const int64_t s = st[order[0]];
    int64_t q = d / s - (d % s < 0 ? 1 : 0);
    for (int i = 0; i < 2; ++i, ++q)
        if (q < a.extent[order[0]] && q > -b.extent[order[0]] && meets(a, b, st, order + 1, n - 1, d - q * s)) return true;
    return false;
}
// Whether the two have a value in common: exact where their strides are the same (views of one
// buffer, as of a projection's output), else only whether they begin at the same address.
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p) return false;
    int64_t enda = a.inner, endb = b.inner, st[3];
    bool same = a.es == b.es;
    int order[3], n = 0;
    for (int i = 0; i < 3; ++i) {
        if (a.extent[i] < 1 || b.extent[i] < 1) return false;
        enda += (a.extent[i] - 1) * a.stride[i];
        endb += (b.extent[i] - 1) * b.stride[i];
        st[i] = a.extent[i] > 1 ? a.stride[i] : b.stride[i];
        same = same && (a.extent[i] < 2 || b.extent[i] < 2 || a.stride[i] == b.stride[i]);
        if ((a.extent[i] < 2 && b.extent[i] < 2) || st[i] == 0) continue;
        int j = n++;
        for (; j > 0 && st[order[j - 1]] < st[i]; --j) order[j] = order[j - 1];
        order[j] = i;
    }
    const char *pa = (const char *)a.p, *pb = (const char *)b.p;
    if (pa == pb) return true;
    if (pa + enda * (int64_t)a.es <= pb || pb + endb * (int64_t)b.es <= pa || !same) return false;
    const int64_t bytes = pb - pa, es = (int64_t)a.es;
    return bytes % es != 0 || meets(a, b, st, order, n, bytes / es);
}
bool same_place(const Span &a, const Span &b) {
    bool same = a.p == b.p;
    for (int i = 0; i < 3; ++i) same = same && (a.extent[i] < 2 || a.stride[i] == b.stride[i]);
    return same;
}
int apart(const Span &out, const Span &in) {
    return overlap(out, in) ? fail(SSM_ERR_ARG, "%s lies over %s", out.name, in.name) : SSM_OK;
}
// the same for two dense arrays of n floats
bool overlap(const float *a, const float *b, size_t n) { return a && b && a < b + n && b < a + n; }

// the same, but each may be the other: rows that lie in one another's place are read before they are
// written, by one team
int apart_or_same(const Span &out, const Span &in) { return same_place(out, in) ? SSM_OK : apart(out, in); }

// ---- rmsnorm -------------------------------------------------------------------------
int check_norm(const ssm_rmsnorm_desc_t *d) {
    if (!d) return fail(SSM_ERR_ARG, "descriptor is NULL");
    if (d->rows < 0) return fail(SSM_ERR_ARG, "rows must be >= 0");
    if (d->dim < 1) return fail(SSM_ERR_ARG, "dim must be >= 1");
    if (!(d->eps >= 0.f) || isinf(d->eps)) return fail(SSM_ERR_ARG, "eps must be finite and >= 0");
    if (d->quant < SSM_QUANT_NONE || d->quant > SSM_QUANT_BLOCK)
        return fail(SSM_ERR_ARG, "unknown quant %d", d->quant);
    if (d->quant == SSM_QUANT_BLOCK && d->dim % 128)
        return fail(SSM_ERR_ARG, "SSM_QUANT_BLOCK needs dim (%lld) to be a multiple of 128",
                    (long long)d->dim);
    if (d->reserved_ != 0) return fail(SSM_ERR_ARG, "reserved descriptor field must be 0");
    if (d->rows > (1ll << 31) - 1 || d->dim > (1 << 20))
        return fail(SSM_ERR_UNSUPPORTED, "rows above 2^31 - 1 or dim above 2^20");
    return check_dtype(d->dtype_io);
}

// ---- rope ----------------------------------------------------------------------------
int check_rope(const ssm_rope_desc_t *d) {
    if (!d) return fail(SSM_ERR_ARG, "descriptor is NULL");
    if (d->batch < 0 || d->seqlen < 0) return fail(SSM_ERR_ARG, "batch and seqlen must be >= 0");
    if (d->nheads_q < 0 || d->nheads_k < 0 || d->headdim < 1)
        return fail(SSM_ERR_ARG, "nheads_q, nheads_k must be >= 0 and headdim >= 1");
    if (d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > d->headdim)
        return fail(SSM_ERR_ARG, "rot_dim (%lld) must be even, >= 2 and <= headdim (%lld)",
                    (long long)d->rot_dim, (long long)d->headdim);
    if (d->layout != SSM_ROPE_HALF && d->layout != SSM_ROPE_PAIRS)
        return fail(SSM_ERR_ARG, "unknown layout %d", d->layout);
    if (!isfinite(d->magnitude)) return fail(SSM_ERR_ARG, "magnitude must be finite");
    if (d->reserved_ != 0) return fail(SSM_ERR_ARG, "reserved descriptor field must be 0");
    if (d->batch > (1 << 24) || d->seqlen > (1ll << 31) - 1 || d->headdim > (1 << 16) ||
        d->nheads_q > (1 << 16) || d->nheads_k > (1 << 16))
        return fail(SSM_ERR_UNSUPPORTED, "sizes exceed the index ranges of the kernels");
    // a thread a value at most
    if ((double)d->batch * (double)d->seqlen * (double)d->headdim > 256.0 * 2147483647.0)
        return fail(SSM_ERR_UNSUPPORTED, "too many tokens for one call");
    return check_dtype(d->dtype_io);
}

int rope(const char *where, const ssm_rope_desc_t *d, const void *q, const void *k,
         const double *freq, const int64_t *positions, void *q_out, void *k_out, float sign,
         void *stream) {
    int rc = check_rope(d);
    if (rc) return rc;
    const int64_t eq[3] = {d->batch, d->seqlen, d->nheads_q}, ek[3] = {d->batch, d->seqlen, d->nheads_k};
    const bool has_q = q != nullptr && d->nheads_q > 0, has_k = k != nullptr && d->nheads_k > 0;
    if ((rc = check_strides3("q", d->stride_q, eq, d->headdim, false)) ||
        (rc = check_strides3("k", d->stride_k, ek, d->headdim, false)) ||
        (has_q && (rc = check_strides3("q_out", d->stride_q_out, eq, d->headdim, true))) ||
        (has_k && (rc = check_strides3("k_out", d->stride_k_out, ek, d->headdim, true))))
        return rc;
    if (d->stride_pos[0] < 0 || d->stride_pos[1] < 0) return fail(SSM_ERR_ARG, "negative stride");
    if (d->batch == 0 || d->seqlen == 0 || (d->nheads_q == 0 && d->nheads_k == 0)) return SSM_OK;
    if (!q && !k) return fail(SSM_ERR_ARG, "q and k are both NULL");
    const size_t es = esize(d->dtype_io);
    if ((has_q && ((rc = need(q, "q", es)) || (rc = need(q_out, "q_out", es)))) ||
        (has_k && ((rc = need(k, "k", es)) || (rc = need(k_out, "k_out", es)))) ||
        (rc = need(freq, "freq", 8)) || (rc = may(positions, "positions", 8)))
        return rc;
    if (!has_q && !has_k) return SSM_OK;
    const Span sq = {"q", has_q ? q : nullptr, d->stride_q, eq, d->headdim, es},
               sk = {"k", has_k ? k : nullptr, d->stride_k, ek, d->headdim, es},
               oq = {"q_out", has_q ? q_out : nullptr, d->stride_q_out, eq, d->headdim, es},
               ok = {"k_out", has_k ? k_out : nullptr, d->stride_k_out, ek, d->headdim, es};
    if ((rc = apart_or_same(oq, sq)) || (rc = apart_or_same(ok, sk)) || (rc = apart(oq, sk)) || (rc = apart(ok, sq)) || (rc = apart(oq, ok)))
        return rc;
    return launched(where, stream, [&](cudaStream_t st) {
        return ssm::rope_rotate(*d, has_q ? q : nullptr, has_k ? k : nullptr, freq, positions, q_out,
                                k_out, sign, st);
    });
}

// ---- linear attention ----------------------------------------------------------------
int check_la(const ssm_linattn_desc_t *d) {
    if (!d) return fail(SSM_ERR_ARG, "descriptor is NULL");
    if (d->batch < 0 || d->seqlen < 0) return fail(SSM_ERR_ARG, "batch and seqlen must be >= 0");
    if (d->nheads < 1 || d->nheads_kv < 1 || d->nheads % d->nheads_kv)
        return fail(SSM_ERR_ARG, "nheads (%lld) must be a multiple of nheads_kv (%lld), both >= 1",
                    (long long)d->nheads, (long long)d->nheads_kv);
    if (d->dim_k < 1 || d->dim_v < 1) return fail(SSM_ERR_ARG, "dim_k and dim_v must be >= 1");
    if (d->route != SSM_LINATTN_AUTO && d->route != SSM_LINATTN_RECURRENT)
        return fail(SSM_ERR_ARG, "unknown route %d", d->route);
    if (d->reserved_ != 0) return fail(SSM_ERR_ARG, "reserved descriptor field must be 0");
    if (d->dim_k > ssm::LA_MAX_DIM || d->dim_v > ssm::LA_MAX_DIM)
        return fail(SSM_ERR_UNSUPPORTED, "dim_k %lld / dim_v %lld above %d", (long long)d->dim_k,
                    (long long)d->dim_v, ssm::LA_MAX_DIM);
    if (d->seqlen > (1ll << 31) - 1 - 256 || d->batch > 65535 || d->nheads > 65535 ||
        d->batch * d->nheads > (1ll << 26))
        return fail(SSM_ERR_UNSUPPORTED, "sizes exceed the index ranges of the kernels");
    const int64_t eh[3] = {d->batch, d->seqlen, d->nheads}, eg[3] = {d->batch, d->seqlen, d->nheads_kv};
    int rc = check_dtype(d->dtype_io);
    if (rc || (rc = check_strides3("q", d->stride_q, eh, d->dim_k, false)) ||
        (rc = check_strides3("k", d->stride_k, eg, d->dim_k, false)) ||
        (rc = check_strides3("v", d->stride_v, eg, d->dim_v, false)) ||
        (rc = check_strides3("o", d->stride_o, eh, d->dim_v, false)) ||
        (rc = check_strides3("dq", d->stride_dq, eh, d->dim_k, false)) ||
        (rc = check_strides3("dk", d->stride_dk, eg, d->dim_k, false)) ||
        (rc = check_strides3("dv", d->stride_dv, eg, d->dim_v, false)))
        return rc;
    return SSM_OK;
}

int la_inputs(const ssm_linattn_desc_t *d, const void *q, const void *k, const void *v,
              const float *log_decay) {
    const size_t es = esize(d->dtype_io);
    int rc;
    if ((rc = need(q, "q", es)) || (rc = need(k, "k", es)) || (rc = need(v, "v", es)) ||
        (rc = need(log_decay, "log_decay", 4)))
        return rc;
    return SSM_OK;
}

// `out` lies over none of the call's inputs (do_ may be null)
int la_apart(const ssm_linattn_desc_t *d, const void *q, const void *k, const void *v, const void *do_, const Span &out) {
    const int64_t eh[3] = {d->batch, d->seqlen, d->nheads}, eg[3] = {d->batch, d->seqlen, d->nheads_kv};
    int rc;
    if ((rc = apart(out, {"q", q, d->stride_q, eh, d->dim_k, out.es})) || (rc = apart(out, {"k", k, d->stride_k, eg, d->dim_k, out.es})) ||
        (rc = apart(out, {"v", v, d->stride_v, eg, d->dim_v, out.es})) || (rc = apart(out, {"do", do_, d->stride_o, eh, d->dim_v, out.es})))
        return rc;
    return SSM_OK;
}
size_t state_floats(const ssm_linattn_desc_t *d) { return (size_t)(d->batch * d->nheads * d->dim_k * d->dim_v); }

// copy of a state, or zeros
cudaError_t state_copy(float *dst, const float *src, const ssm_linattn_desc_t *d, cudaStream_t st) {
    const size_t n = sizeof(float) * state_floats(d);
    if (!dst || dst == src || n == 0) return cudaSuccess;
    return src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, st)
               : cudaMemsetAsync(dst, 0, n, st);
}

struct Operand {
    const void *p;
    const int64_t *s;
    int rep, dim;
};
// the walk whose output pairs `a` with the state of (k, v); `flip`: the state is kept
// transposed to [dim_k][dim_v]
LaWalk walk(Operand a, Operand k, Operand v, void *o, const int64_t *so, const float *s_in,
            float *s_out, bool flip, float read, float write, bool rev) {
    LaWalk w = {};
    w.a = a.p;
    w.k = k.p;
    w.v = v.p;
    w.o = o;
    for (int i = 0; i < 3; ++i) {
        w.sa[i] = a.s[i];
        w.sk[i] = k.s[i];
        w.sv[i] = v.s[i];
        w.so[i] = so ? so[i] : 0;
    }
    w.rep_a = a.rep;
    w.rep_k = k.rep;
    w.rep_v = v.rep;
    w.da = a.dim;
    w.dc = v.dim;
    w.s_in = s_in;
    w.s_out = s_out;
    w.st_a = flip ? 1 : v.dim;
    w.st_c = flip ? a.dim : 1;
    w.read = read;
    w.write = write;
    w.rev = rev;
    return w;
}

LaArgs la_args(const ssm_linattn_desc_t *d, const float *log_decay, const int32_t *lengths) {
    LaArgs p = {};
    p.B = (int)d->batch;
    p.L = (int)d->seqlen;
    p.H = (int)d->nheads;
    p.bf16 = d->dtype_io == SSM_BF16;
    p.log_decay = log_decay;
    p.lengths = lengths;
    return p;
}

// Workspace of a call: per-head dk and dv of the backward where heads share a key and value
// head, and the segment states of its walks on tensor cores.
struct LaWs {
    int nseg;   // 0: the recurrence
    size_t dk, dv, seg[3], total;
};
LaWs la_layout(const ssm_linattn_desc_t *d, bool bwd) {
    LaWs w = {};
    const int ndk = (int)d->dim_k, ndv = (int)d->dim_v;
    if (bwd && d->nheads != d->nheads_kv) {
        const size_t tok = (size_t)(d->batch * d->seqlen * d->nheads);
        w.dv = align256(tok * ndk * 4);
        w.total = w.dv + align256(tok * ndv * 4);
    }
    if (d->route != SSM_LINATTN_AUTO) return w;
    // A block on tensor cores takes 10 us whatever it walks, a token of the recurrence 0.1 to 0.4 us:
    // on one B200, 4 batch rows of 16 heads of 64 took 6.3 us for 32 tokens by the latter and
    // 10.5 us by the former, and 10.1 and 10.4 us for 64 (the gradient 12.4 and 17.7, 20.6 and 17.7);
    // heads of 128 8.9 and 10.9 us for 16 tokens, 14.4 and 10.9 us for 32 (26.4 and 26.0, 40.6 and 25.9).
    if (d->seqlen * (d->dim_k > d->dim_v ? d->dim_k : d->dim_v) <= 2048) return w;
    const bool bf16 = d->dtype_io == SSM_BF16;
    if (!ssm::la_chunked_sizes(bf16, ndk, ndv) || (bwd && !ssm::la_chunked_sizes(bf16, ndv, ndk))) return w;
    const int sk = (ndk + 63) / 64, sv = (ndv + 63) / 64;   // 64-column slices
    w.nseg = ssm::la_segments(d->seqlen, d->batch * d->nheads * (bwd ? 2 * sk + sv : sv));
    if (w.nseg > 1)
        for (int i = 0; i < (bwd ? 3 : 1); ++i) {
            w.seg[i] = w.total;
            w.total += align256((size_t)w.nseg * (size_t)(d->batch * d->nheads * ndk * ndv) * 4);
        }
    return w;
}

// the walks of `p` on tensor cores where they apply, else by the recurrence
cudaError_t la_run(const LaArgs &p, const LaWs &ws, void *workspace, cudaStream_t st) {
    if (ws.nseg) {
        float *seg[3];
        for (int i = 0; i < 3; ++i) seg[i] = (float *)((char *)workspace + ws.seg[i]);
        cudaError_t e;
        if (ssm::la_chunked(p, ws.nseg, seg, st, &e)) return e;
    }
    return ssm::la_recurrent(p, st);
}

int la_workspace(const char *where, size_t want, const void *ws, size_t bytes) {
    if (want && (!ws || bytes < want))
        return fail(SSM_ERR_WORKSPACE, "%s needs a workspace of %zu bytes", where, want);
    if (want && (uintptr_t)ws % 256) return fail(SSM_ERR_ALIGN, "workspace is not 256-byte aligned");
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_rmsnorm_fwd(const ssm_rmsnorm_desc_t *d, const void *x, const void *residual,
                    const float *weight, void *r, void *y, void *y8, float *scales, float *rstd,
                    void *stream) {
    int rc = check_norm(d);
    if (rc) return rc;
    const bool q = d->quant != SSM_QUANT_NONE;
    if ((rc = check_stride("x", d->stride_x, d->rows, d->dim, false)) ||
        (rc = check_stride("residual", d->stride_residual, d->rows, d->dim, false)) ||
        (r && (rc = check_stride("r", d->stride_r, d->rows, d->dim, true))) ||
        (y && (rc = check_stride("y", d->stride_y, d->rows, d->dim, true))) ||
        (q && (rc = check_stride("y8", d->stride_y8, d->rows, d->dim, true))))
        return rc;
    if (d->rows == 0) return SSM_OK;
    const size_t es = esize(d->dtype_io);
    if ((rc = need(x, "x", es)) || (rc = may(residual, "residual", es)) ||
        (rc = may(weight, "weight", 4)) || (rc = residual ? need(r, "r", es) : may(r, "r", es)) ||
        (rc = q ? may(y, "y", es) : need(y, "y", es)) || (rc = may(rstd, "rstd", 4)))
        return rc;
    if (q && ((rc = need(y8, "y8", 1)) || (rc = need(scales, "scales", 4)))) return rc;
    const int64_t rows[3] = {d->rows, 1, 1}, ix[3] = {d->stride_x}, ires[3] = {d->stride_residual}, ir[3] = {d->stride_r},
                  iy[3] = {d->stride_y};
    const Span sx = {"x", x, ix, rows, d->dim, es}, sres = {"residual", residual, ires, rows, d->dim, es},
               sr = {"r", r, ir, rows, d->dim, es}, sy = {"y", y, iy, rows, d->dim, es};
    if ((rc = apart_or_same(sr, sx)) || (rc = apart_or_same(sr, sres)) || (rc = apart_or_same(sy, sx)) ||
        (rc = apart_or_same(sy, sres)) || (rc = apart(sy, sr)))
        return rc;
    return launched("ssm_rmsnorm_fwd", stream, [&](cudaStream_t st) {
        return ssm::rmsnorm_forward(*d, x, residual, weight, r, y, q ? y8 : nullptr, scales, rstd, st);
    });
}

size_t ssm_rmsnorm_workspace_size(const ssm_rmsnorm_desc_t *d) {
    if (check_norm(d) != SSM_OK || d->rows == 0) return 0;
    return ssm::rmsnorm_bwd_bytes(*d);
}

int ssm_rmsnorm_bwd(const ssm_rmsnorm_desc_t *d, const void *dy, const void *r, const float *weight,
                    const float *rstd, const void *dr, void *dx, float *dweight, void *workspace,
                    size_t workspace_bytes, void *stream) {
    int rc = check_norm(d);
    if (rc) return rc;
    if ((rc = check_stride("dy", d->stride_dy, d->rows, d->dim, false)) ||
        (rc = check_stride("r", d->stride_r, d->rows, d->dim, false)) ||
        (rc = check_stride("dr", d->stride_dr, d->rows, d->dim, false)) ||
        (rc = check_stride("dx", d->stride_dx, d->rows, d->dim, true)))
        return rc;
    if ((rc = may(dweight, "dweight", 4))) return rc;
    if (d->rows == 0) {
        if (!dweight) return SSM_OK;
        return launched("ssm_rmsnorm_bwd (empty)", stream, [&](cudaStream_t st) {
            return cudaMemsetAsync(dweight, 0, sizeof(float) * d->dim, st);
        });
    }
    const size_t es = esize(d->dtype_io);
    if ((rc = need(dy, "dy", es)) || (rc = need(r, "r", es)) || (rc = may(weight, "weight", 4)) ||
        (rc = need(rstd, "rstd", 4)) || (rc = may(dr, "dr", es)) || (rc = need(dx, "dx", es)))
        return rc;
    if (dweight && (rc = la_workspace("ssm_rmsnorm_bwd", ssm::rmsnorm_bwd_bytes(*d), workspace,
                                      workspace_bytes)))
        return rc;
    const int64_t rows[3] = {d->rows, 1, 1}, idy[3] = {d->stride_dy}, ir[3] = {d->stride_r}, idr[3] = {d->stride_dr},
                  idx[3] = {d->stride_dx};
    const Span sdx = {"dx", dx, idx, rows, d->dim, es};
    if ((rc = apart_or_same(sdx, {"dy", dy, idy, rows, d->dim, es})) || (rc = apart_or_same(sdx, {"r", r, ir, rows, d->dim, es})) ||
        (rc = apart_or_same(sdx, {"dr", dr, idr, rows, d->dim, es})))
        return rc;
    return launched("ssm_rmsnorm_bwd", stream, [&](cudaStream_t st) {
        return ssm::rmsnorm_backward(*d, dy, r, weight, rstd, dr, dx, dweight, (float *)workspace, st);
    });
}

int ssm_rope_frequencies(int64_t rot_dim, double base, int scaling, double factor, double low_turns,
                         double high_turns, double original_context, double *freq) {
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > (1 << 16))
        return fail(SSM_ERR_ARG, "rot_dim (%lld) must be even and in 2 .. 65536", (long long)rot_dim);
    if (!(base > 0) || isinf(base)) return fail(SSM_ERR_ARG, "base must be positive");
    if (scaling < SSM_ROPE_PLAIN || scaling > SSM_ROPE_BANDS)
        return fail(SSM_ERR_ARG, "unknown scaling %d", scaling);
    if (scaling != SSM_ROPE_PLAIN && (!(factor >= 1) || isinf(factor)))
        return fail(SSM_ERR_ARG, "factor must be finite and >= 1");
    if (scaling == SSM_ROPE_NTK && rot_dim < 4)
        return fail(SSM_ERR_ARG, "SSM_ROPE_NTK needs rot_dim >= 4");
    if (scaling == SSM_ROPE_BANDS &&
        !(low_turns >= 0 && low_turns < high_turns && original_context > 0 && isfinite(high_turns) &&
          isfinite(original_context)))
        return fail(SSM_ERR_ARG, "SSM_ROPE_BANDS needs 0 <= low_turns < high_turns and original_context > 0");
    if (!freq) return fail(SSM_ERR_ARG, "freq is NULL");
    const double d = (double)rot_dim;
    const double b = scaling == SSM_ROPE_NTK ? base * pow(factor, d / (d - 2)) : base;
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double f = pow(b, -2.0 * (double)i / d);
        if (scaling == SSM_ROPE_LINEAR) f /= factor;
        if (scaling == SSM_ROPE_BANDS) {
            const double turns = original_context * f / (2.0 * M_PI);
            double keep = (turns - low_turns) / (high_turns - low_turns);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = keep * f + (1 - keep) * f / factor;
        }
        freq[i] = f;
    }
    ssm::abi_ok();
    return SSM_OK;
}

int ssm_rope_fwd(const ssm_rope_desc_t *d, const void *q, const void *k, const double *freq,
                 const int64_t *positions, void *q_out, void *k_out, void *stream) {
    return rope("ssm_rope_fwd", d, q, k, freq, positions, q_out, k_out, 1.f, stream);
}

int ssm_rope_bwd(const ssm_rope_desc_t *d, const void *dq, const void *dk, const double *freq,
                 const int64_t *positions, void *dq_out, void *dk_out, void *stream) {
    return rope("ssm_rope_bwd", d, dq, dk, freq, positions, dq_out, dk_out, -1.f, stream);
}

size_t ssm_linattn_workspace_size(const ssm_linattn_desc_t *d, int pass) {
    if (check_la(d) != SSM_OK || d->batch == 0 || d->seqlen == 0) return 0;
    return pass == SSM_PASS_BWD || pass == SSM_PASS_FWD ? la_layout(d, pass == SSM_PASS_BWD).total : 0;
}

int ssm_linattn_fwd(const ssm_linattn_desc_t *d, const void *q, const void *k, const void *v,
                    const float *log_decay, const float *state_in, const int32_t *lengths, void *o,
                    float *state_out, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_la(d);
    if (rc) return rc;
    const int64_t eh[3] = {d->batch, d->seqlen, d->nheads};
    if (o && (rc = check_strides3("o", d->stride_o, eh, d->dim_v, true))) return rc;
    const bool empty = d->batch == 0 || d->seqlen == 0;
    if (!o && !state_out && !empty) return fail(SSM_ERR_ARG, "o and state_out are both NULL");
    if ((rc = may(state_in, "state_in", 4)) || (rc = may(state_out, "state_out", 4)) ||
        (rc = may(lengths, "lengths", 4)) || (rc = may(o, "o", esize(d->dtype_io))))
        return rc;
    if (state_out != state_in && overlap(state_out, state_in, state_floats(d)))
        return fail(SSM_ERR_ARG, "state_out lies over a part of state_in");
    if (empty)
        return launched("ssm_linattn_fwd (empty)", stream,
                        [&](cudaStream_t st) { return state_copy(state_out, state_in, d, st); });
    if ((rc = la_inputs(d, q, k, v, log_decay))) return rc;
    const LaWs ws = la_layout(d, false);
    if ((rc = la_workspace("ssm_linattn_fwd", ws.total, workspace, workspace_bytes))) return rc;
    if ((rc = la_apart(d, q, k, v, nullptr, {"o", o, d->stride_o, eh, d->dim_v, esize(d->dtype_io)}))) return rc;
    const int rep = (int)(d->nheads / d->nheads_kv), dk = (int)d->dim_k, dv = (int)d->dim_v;
    LaArgs p = la_args(d, log_decay, lengths);
    p.nwalk = 1;
    p.w[0] = walk({q, d->stride_q, 1, dk}, {k, d->stride_k, rep, dk}, {v, d->stride_v, rep, dv}, o,
                  d->stride_o, state_in, state_out, false, d->scale, 1.f, false);
    return launched("ssm_linattn_fwd", stream,
                    [&](cudaStream_t st) { return la_run(p, ws, workspace, st); });
}

int ssm_linattn_bwd(const ssm_linattn_desc_t *d, const void *q, const void *k, const void *v,
                    const float *log_decay, const float *state_in, const int32_t *lengths,
                    const void *do_, const float *dstate_out, void *dq, void *dk, void *dv,
                    float *dstate_in, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_la(d);
    if (rc) return rc;
    const int64_t eh[3] = {d->batch, d->seqlen, d->nheads}, eg[3] = {d->batch, d->seqlen, d->nheads_kv};
    if ((rc = check_strides3("dq", d->stride_dq, eh, d->dim_k, true)) ||
        (rc = check_strides3("dk", d->stride_dk, eg, d->dim_k, true)) ||
        (rc = check_strides3("dv", d->stride_dv, eg, d->dim_v, true)))
        return rc;
    if ((rc = may(state_in, "state_in", 4)) || (rc = may(dstate_out, "dstate_out", 4)) ||
        (rc = may(dstate_in, "dstate_in", 4)) || (rc = may(lengths, "lengths", 4)))
        return rc;
    if (dstate_in && (dstate_in == dstate_out || dstate_in == state_in))
        return fail(SSM_ERR_ARG, "dstate_in must be neither dstate_out nor state_in");
    const bool over = overlap(dstate_in, dstate_out, state_floats(d)) || overlap(dstate_in, state_in, state_floats(d));
    if (!over && (d->batch == 0 || d->seqlen == 0))
        return launched("ssm_linattn_bwd (empty)", stream,
                        [&](cudaStream_t st) { return state_copy(dstate_in, dstate_out, d, st); });
    const size_t es = esize(d->dtype_io);
    if ((rc = la_inputs(d, q, k, v, log_decay)) || (rc = need(do_, "do", es)) ||
        (rc = need(dq, "dq", es)) || (rc = need(dk, "dk", es)) || (rc = need(dv, "dv", es)))
        return rc;
    const LaWs ws = la_layout(d, true);
    if ((rc = la_workspace("ssm_linattn_bwd", ws.total, workspace, workspace_bytes))) return rc;
    const Span sdq = {"dq", dq, d->stride_dq, eh, d->dim_k, es}, sdk = {"dk", dk, d->stride_dk, eg, d->dim_k, es},
               sdv = {"dv", dv, d->stride_dv, eg, d->dim_v, es};
    if ((rc = la_apart(d, q, k, v, do_, sdq)) || (rc = la_apart(d, q, k, v, do_, sdk)) ||
        (rc = la_apart(d, q, k, v, do_, sdv)) || (rc = apart(sdq, sdk)) || (rc = apart(sdq, sdv)) || (rc = apart(sdk, sdv)))
        return rc;
    if (over) return fail(SSM_ERR_ARG, "dstate_in lies over a part of dstate_out or state_in");
    const int rep = (int)(d->nheads / d->nheads_kv), ndk = (int)d->dim_k, ndv = (int)d->dim_v;
    const Operand oq = {q, d->stride_q, 1, ndk}, ok = {k, d->stride_k, rep, ndk},
                  ov = {v, d->stride_v, rep, ndv}, odo = {do_, d->stride_o, 1, ndv};
    // shared key and value heads: the gradients of every head first, fp32 and dense
    const int64_t L = d->seqlen, H = d->nheads;
    const int64_t hk[3] = {L * H * ndk, H * ndk, ndk}, hv[3] = {L * H * ndv, H * ndv, ndv};
    const bool shared = rep > 1;
    char *base = (char *)workspace;
    void *tk = shared ? base + ws.dk : dk, *tv = shared ? base + ws.dv : dv;
    LaArgs p = la_args(d, log_decay, lengths);
    p.nwalk = 3;
    p.w[0] = walk(odo, ov, ok, dq, d->stride_dq, state_in, nullptr, true, d->scale, 1.f, false);
    p.w[1] = walk(ov, odo, oq, tk, shared ? hk : d->stride_dk, dstate_out, nullptr, true, 1.f, d->scale, true);
    p.w[2] = walk(ok, oq, odo, tv, shared ? hv : d->stride_dv, dstate_out, dstate_in, false, 1.f, d->scale, true);
    p.w[1].o_f32 = p.w[2].o_f32 = shared;
    return launched("ssm_linattn_bwd", stream, [&](cudaStream_t st) {
        cudaError_t e = la_run(p, ws, workspace, st);
        if (e != cudaSuccess || !shared) return e;
        const long long sk[3] = {d->stride_dk[0], d->stride_dk[1], d->stride_dk[2]};
        const long long sv[3] = {d->stride_dv[0], d->stride_dv[1], d->stride_dv[2]};
        if ((e = ssm::la_group_sum((const float *)tk, dk, sk, p.B, p.L, p.H, rep, ndk, lengths, p.bf16, st)))
            return e;
        return ssm::la_group_sum((const float *)tv, dv, sv, p.B, p.L, p.H, rep, ndv, lengths, p.bf16, st);
    });
}

int ssm_linattn_step(const ssm_linattn_desc_t *d, const void *q, const void *k, const void *v,
                     const float *log_decay, float *state, void *o, void *stream) {
    int rc = check_la(d);
    if (rc) return rc;
    if (d->seqlen != 1)
        return fail(SSM_ERR_ARG, "ssm_linattn_step takes one token (seqlen %lld)", (long long)d->seqlen);
    const int64_t eh[3] = {d->batch, 1, d->nheads};
    if ((rc = check_strides3("o", d->stride_o, eh, d->dim_v, true))) return rc;
    if (d->batch == 0) return SSM_OK;
    if ((rc = la_inputs(d, q, k, v, log_decay)) || (rc = need(state, "state", 4)) ||
        (rc = need(o, "o", esize(d->dtype_io))) ||
        (rc = la_apart(d, q, k, v, nullptr, {"o", o, d->stride_o, eh, d->dim_v, esize(d->dtype_io)})))
        return rc;
    return launched("ssm_linattn_step", stream, [&](cudaStream_t st) {
        return ssm::la_step(*d, q, k, v, log_decay, state, o, st);
    });
}

}  // extern "C"
