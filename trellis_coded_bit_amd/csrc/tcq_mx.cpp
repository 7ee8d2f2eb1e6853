// libtcq C ABI of the microscaled operators: argument checks and workspace sizes.  The numeric
// steps run in kernels_mx.hip and kernels_mx_linear.hip.
#include "tcq.h"
#include "abi_checks.h"
#include "region.h"
#include "tcq_internal.h"

using namespace tcq;

namespace {

int64_t groups_of(int64_t n) { return (n + 31) / 32; }

int64_t row_bytes(int format, int64_t cols) {
    return groups_of(cols) * (format == TCQ_FP4 ? 16 : 32);
}

int check_mx_shape(const char *fn, int format, int dtype, int64_t rows, int64_t cols) {
    int rc = check_format(fn, format);
    if (rc == TCQ_OK) rc = check_dtype(fn, dtype);
    if (rc != TCQ_OK) return rc;
    if (rows < 0 || cols < 0) {
        set_error("%s: negative size (rows=%lld cols=%lld)", fn, (long long)rows,
                  (long long)cols);
        return TCQ_EINVAL;
    }
    if (rows > 0x7FFFFFFF || cols > 0x7FFFFFFF) {
        set_error("%s: rows=%lld, cols=%lld above 2^31 - 1", fn, (long long)rows,
                  (long long)cols);
        return TCQ_EUNSUPPORTED;
    }
    return TCQ_OK;
}

// Codes of a matrix: rows of whole groups, on 16 bytes.
int check_codes(const char *fn, const char *name, const uint8_t *codes, int64_t ld,
                const uint8_t *scale, int format, int64_t cols) {
    if (!codes || !scale) {
        set_error("%s: %s's codes and scale bytes must be non-NULL", fn, name);
        return TCQ_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(codes) % 16 || ld % 16) {
        set_error("%s: %s's rows of codes start on multiples of 16 bytes (address %p, leading "
                  "dimension %lld)", fn, name, static_cast<const void *>(codes), (long long)ld);
        return TCQ_EINVAL;
    }
    if (ld < row_bytes(format, cols)) {
        set_error("%s: leading dimension %lld of %s's codes is below %lld bytes (whole groups)",
                  fn, (long long)ld, name, (long long)row_bytes(format, cols));
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

Region codes_region(const char *name, const uint8_t *codes, int64_t rows, int64_t ld, int format,
                    int64_t cols) {
    return region(name, codes, rows, ld, row_bytes(format, cols), 1);
}
Region scale_region(const char *name, const uint8_t *scale, int64_t rows, int64_t cols) {
    return region(name, scale, 1, 0, rows * groups_of(cols), 1);
}

int check_mx_layer(const char *fn, int format, int dtype, int64_t B, int64_t M, int64_t N) {
    int rc = check_format(fn, format);
    if (rc == TCQ_OK) rc = check_dtype(fn, dtype);
    if (rc != TCQ_OK) return rc;
    if (B < 0 || M < 0 || N < 0) {
        set_error("%s: negative size (B=%lld M=%lld N=%lld)", fn, (long long)B, (long long)M,
                  (long long)N);
        return TCQ_EINVAL;
    }
    if (M > TCQ_LINEAR_MAX_DIM || N > TCQ_LINEAR_MAX_DIM || B > TCQ_LINEAR_MAX_BATCH) {
        set_error("%s: outside the layer's limits (M, N <= %d, B <= %d): B=%lld M=%lld N=%lld",
                  fn, TCQ_LINEAR_MAX_DIM, TCQ_LINEAR_MAX_BATCH, (long long)B, (long long)M,
                  (long long)N);
        return TCQ_EUNSUPPORTED;
    }
    return TCQ_OK;
}

}  // namespace

extern "C" int tcq_mx_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int format, uint8_t *codes, int64_t ldq, uint8_t *scale,
                           hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_mx_pack";
    int rc = check_mx_shape(fn, format, dtype, rows, cols);
    if (rc != TCQ_OK) return rc;
    if (rows == 0 || cols == 0) return TCQ_OK;
    rc = check_matrix(fn, "X", X, ldx, cols, size_of(dtype));
    if (rc == TCQ_OK) rc = check_codes(fn, "the result", codes, ldq, scale, format, cols);
    if (rc != TCQ_OK) return rc;
    const Region rX = region("X", X, rows, ldx, cols, size_of(dtype));
    const Region rq = codes_region("codes", codes, rows, ldq, format, cols);
    const Region rs = scale_region("scale", scale, rows, cols);
    rc = check_apart(fn, rq, rX);
    if (rc == TCQ_OK) rc = check_apart(fn, rs, rX);
    if (rc == TCQ_OK) rc = check_apart(fn, rs, rq);
    if (rc != TCQ_OK) return rc;
    const hipError_t e = launch_mx_pack(X, dtype, rows, cols, ldx, format, codes, ldq, scale,
                                        nullptr, 0, nullptr, stream);
    if (e != hipSuccess) return hip_fail(fn, "quantisation launch", e);
    return TCQ_OK;
}

extern "C" int tcq_mx_unpack(const uint8_t *codes, int64_t ldq, const uint8_t *scale,
                             int64_t rows, int64_t cols, int format, int dtype, void *out,
                             int64_t ldo, hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_mx_unpack";
    int rc = check_mx_shape(fn, format, dtype, rows, cols);
    if (rc != TCQ_OK) return rc;
    if (rows == 0 || cols == 0) return TCQ_OK;
    rc = check_codes(fn, "the input", codes, ldq, scale, format, cols);
    if (rc == TCQ_OK) rc = check_matrix(fn, "out", out, ldo, cols, size_of(dtype));
    if (rc != TCQ_OK) return rc;
    const Region ro = region("out", out, rows, ldo, cols, size_of(dtype));
    rc = check_apart(fn, ro, codes_region("codes", codes, rows, ldq, format, cols));
    if (rc == TCQ_OK) rc = check_apart(fn, ro, scale_region("scale", scale, rows, cols));
    if (rc != TCQ_OK) return rc;
    const hipError_t e = launch_mx_unpack(MxMatrix{codes, ldq, scale, format}, rows, cols, dtype,
                                          out, ldo, cols, stream);
    if (e != hipSuccess) return hip_fail(fn, "unpacking launch", e);
    return TCQ_OK;
}

extern "C" int tcq_mx_linear_workspace_bytes(int format, int64_t B, int64_t M, int64_t N,
                                             size_t *bytes) {
    clear_error();
    const char *fn = "tcq_mx_linear_workspace_bytes";
    const int rc = check_mx_layer(fn, format, TCQ_F32, B, M, N);
    if (rc != TCQ_OK) return rc;
    if (!bytes) {
        set_error("%s: bytes is NULL", fn);
        return TCQ_EINVAL;
    }
    *bytes = B == 0 || M == 0 ? 0 : mx_linear_layout(format, B, M, N).bytes;
    return TCQ_OK;
}

extern "C" int tcq_mx_linear(const uint8_t *w_codes, int64_t ldw, const uint8_t *w_scale,
                             int64_t M, int64_t N, int dtype, const void *x, int64_t B,
                             int64_t ldx, int format, uint8_t *x_codes, int64_t ldxq,
                             uint8_t *x_scale, const float *bias, const void *residual,
                             int64_t ldr, void *y, int64_t ldy, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_mx_linear";
    int rc = check_mx_layer(fn, format, dtype, B, M, N);
    if (rc != TCQ_OK) return rc;
    if (M == 0 || B == 0) return TCQ_OK;
    const size_t size = size_of(dtype);
    const bool keep = x && (x_codes || x_scale);
    if (N > 0) {
        rc = check_codes(fn, "w", w_codes, ldw, w_scale, TCQ_FP4, N);
        if (rc == TCQ_OK && x) rc = check_matrix(fn, "x", x, ldx, N, size);
        if (rc == TCQ_OK && (!x || keep))
            rc = check_codes(fn, "x", x_codes, ldxq, x_scale, format, N);
        if (rc != TCQ_OK) return rc;
    }
    rc = check_matrix(fn, "y", y, ldy, M, size);
    if (rc != TCQ_OK) return rc;
    if (residual) {
        rc = check_matrix(fn, "residual", residual, ldr, M, size);
        if (rc != TCQ_OK) return rc;
        if (residual == y && ldr != ldy) {
            set_error("%s: residual in place of y needs ldr == ldy", fn);
            return TCQ_EINVAL;
        }
    }
    rc = check_workspace(fn, workspace, workspace_bytes, mx_linear_layout(format, B, M, N).bytes);
    if (rc != TCQ_OK) return rc;
    const bool in = N > 0;
    const Region ry = region("y", y, B, ldy, M, size);
    const Region rx = region("x", in ? x : nullptr, B, ldx, N, size);
    const Region rr = region("residual", residual == y ? nullptr : residual, B, ldr, M, size);
    const Region rw = codes_region("w's codes", in ? w_codes : nullptr, M, ldw, TCQ_FP4, N);
    const Region rws = scale_region("w's scale bytes", in ? w_scale : nullptr, M, N);
    const Region rq = codes_region("x's codes", in ? x_codes : nullptr, B, ldxq, format, N);
    const Region rs = scale_region("x's scale bytes", in ? x_scale : nullptr, B, N);
    for (const Region *r : {&rx, &rr, &rw, &rws, &rq, &rs}) {
        rc = check_apart(fn, ry, *r);
        if (rc != TCQ_OK) return rc;
    }
    if (keep) {
        for (const Region *r : {&rx, &rr, &rw, &rws}) {
            rc = check_apart(fn, rq, *r);
            if (rc == TCQ_OK) rc = check_apart(fn, rs, *r);
            if (rc != TCQ_OK) return rc;
        }
        rc = check_apart(fn, rs, rq);
        if (rc != TCQ_OK) return rc;
    }
    const MxLinearCall c{{w_codes, ldw, w_scale, TCQ_FP4}, M, N, x, ldx,
                         {x_codes, ldxq, x_scale, format}, keep, dtype, B, bias, residual, ldr, y,
                         ldy};
    const hipError_t e = launch_mx_linear(c, static_cast<char *>(workspace), stream);
    if (e != hipSuccess) return hip_fail(fn, "linear layer launch", e);
    return TCQ_OK;
}

extern "C" int tcq_mx_linear_backward_workspace_bytes(int dtype, int64_t B, int64_t M, int64_t N,
                                                      int dx, int dw, int dbias, size_t *bytes) {
    clear_error();
    const char *fn = "tcq_mx_linear_backward_workspace_bytes";
    const int rc = check_mx_layer(fn, TCQ_FP4, dtype, B, M, N);
    if (rc != TCQ_OK) return rc;
    if (!bytes) {
        set_error("%s: bytes is NULL", fn);
        return TCQ_EINVAL;
    }
    *bytes = mx_grad_bytes(dtype, B, M, N, dx != 0, dw != 0, dbias != 0);
    return TCQ_OK;
}

extern "C" int tcq_mx_linear_backward(const uint8_t *w_codes, int64_t ldw, const uint8_t *w_scale,
                                      int64_t M, int64_t N, int dtype, const void *dy, int64_t B,
                                      int64_t lddy, int format, const uint8_t *x_codes,
                                      int64_t ldxq, const uint8_t *x_scale, void *dx,
                                      int64_t lddx, void *dw, int64_t lddw, float *dbias,
                                      void *workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_mx_linear_backward";
    int rc = check_mx_layer(fn, format, dtype, B, M, N);
    if (rc != TCQ_OK) return rc;
    if (!dx && !dw && !dbias) {
        set_error("%s: none of dx, dw and dbias is wanted", fn);
        return TCQ_EINVAL;
    }
    const size_t size = size_of(dtype);
    if (B > 0 && M > 0) {
        rc = check_matrix(fn, "dy", dy, lddy, M, size);
        if (rc != TCQ_OK) return rc;
    }
    const bool has_dx = dx && B > 0 && N > 0, has_dw = dw && M > 0 && N > 0;
    if (has_dx) {
        rc = check_matrix(fn, "dx", dx, lddx, N, size);
        if (rc == TCQ_OK && M > 0) rc = check_codes(fn, "w", w_codes, ldw, w_scale, TCQ_FP4, N);
        if (rc != TCQ_OK) return rc;
    }
    if (has_dw) {
        rc = check_matrix(fn, "dw", dw, lddw, N, size);
        if (rc == TCQ_OK && B > 0) rc = check_codes(fn, "x", x_codes, ldxq, x_scale, format, N);
        if (rc != TCQ_OK) return rc;
    }
    rc = check_workspace(fn, workspace, workspace_bytes,
                         mx_grad_bytes(dtype, B, M, N, dx != nullptr, dw != nullptr,
                                       dbias != nullptr));
    if (rc != TCQ_OK) return rc;
    const Region out[3] = {region("dx", has_dx ? dx : nullptr, B, lddx, N, size),
                           region("dw", has_dw ? dw : nullptr, M, lddw, N, size),
                           region("dbias", dbias, 1, 0, M, sizeof(float))};
    const Region in[5] = {
        region("dy", dy, B, lddy, M, size),
        codes_region("w's codes", has_dx ? w_codes : nullptr, M, ldw, TCQ_FP4, N),
        scale_region("w's scale bytes", has_dx ? w_scale : nullptr, M, N),
        codes_region("x's codes", has_dw ? x_codes : nullptr, B, ldxq, format, N),
        scale_region("x's scale bytes", has_dw ? x_scale : nullptr, B, N)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j) {
            rc = check_apart(fn, out[i], out[j]);
            if (rc != TCQ_OK) return rc;
        }
        for (const Region &r : in) {
            rc = check_apart(fn, out[i], r);
            if (rc != TCQ_OK) return rc;
        }
    }
    const MxGrad c{dtype, dy, B, lddy, M, N, {w_codes, ldw, w_scale, TCQ_FP4},
                   {x_codes, ldxq, x_scale, format}, dx, lddx, dw, lddw, dbias};
    const hipError_t e = launch_mx_grad(c, static_cast<char *>(workspace), stream);
    if (e != hipSuccess) return hip_fail(fn, "linear layer gradient launch", e);
    return TCQ_OK;
}
