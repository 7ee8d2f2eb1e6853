// libtcq C ABI of the coded linear layer and the 8-bit checkpoints: argument checks and
// workspace sizes.  The numeric steps run in kernels_linear.hip and kernels_checkpoint.hip.
#include "tcq.h"
#include "abi_checks.h"
#include "region.h"
#include "tcq_internal.h"

using namespace tcq;

namespace {

int check_act(const char *fn, int act) {
    if (act < TCQ_ACT_NONE || act > TCQ_ACT_GELU) {
        set_error("%s: act=%d is no activation of tcq_act", fn, act);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

int check_layer(const char *fn, int dtype, int64_t B, int64_t M, int64_t N, int L, int k, int V,
                int T) {
    int rc = check_trellis(fn, M, N, L, k, V, T);
    if (rc != TCQ_OK) return rc;
    rc = check_dtype(fn, dtype);
    if (rc != TCQ_OK) return rc;
    if (B < 0) {
        set_error("%s: negative batch B=%lld", fn, (long long)B);
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

int check_coded(const char *fn, const void *bits, const void *s0, const void *table,
                size_t size) {
    if (!bits || !s0 || !table) {
        set_error("%s: bitstream, start_state and codebook must be non-NULL", fn);
        return TCQ_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(table) % size) {
        set_error("%s: codebook at %p is not aligned to its values of %zu bytes", fn, table,
                  size);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

size_t forward_bytes(int dtype, int64_t B, int64_t M, int64_t N, int L, int k, int V, int T) {
    const int bt = linear_small(size_of(dtype), B, N, L, k, V, T);
    return bt ? linear_small_bytes(size_of(dtype), N, bt)
              : linear_layout(size_of(dtype), B, M, N).bytes;
}

int check_pack(const char *fn, int dtype, int64_t rows, int64_t cols) {
    const int rc = check_dtype(fn, dtype);
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

}  // namespace

extern "C" int tcq_decode_linear_workspace_bytes(int dtype, int64_t B, int64_t M, int64_t N,
                                                 int L, int k, int V, int T, size_t *bytes) {
    clear_error();
    const char *fn = "tcq_decode_linear_workspace_bytes";
    const int rc = check_layer(fn, dtype, B, M, N, L, k, V, T);
    if (rc != TCQ_OK) return rc;
    if (!bytes) {
        set_error("%s: bytes is NULL", fn);
        return TCQ_EINVAL;
    }
    *bytes = (B == 0 || M == 0) ? 0 : forward_bytes(dtype, B, M, N, L, k, V, T);
    return TCQ_OK;
}

extern "C" int tcq_decode_linear(const uint32_t *bitstream, const uint32_t *start_state,
                                 const void *codebook, int64_t M, int64_t N, int L, int k,
                                 int V, int T, int dtype, const void *x, int64_t B,
                                 int64_t ldx, const float *row_scale, const float *bias,
                                 int act, const void *residual, int64_t ldr, void *y,
                                 int64_t ldy, void *pre, int64_t ldp, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_decode_linear";
    int rc = check_layer(fn, dtype, B, M, N, L, k, V, T);
    if (rc != TCQ_OK) return rc;
    rc = check_act(fn, act);
    if (rc != TCQ_OK) return rc;
    if (M == 0 || B == 0) return TCQ_OK;
    const size_t size = size_of(dtype);
    if (N > 0) {
        rc = check_coded(fn, bitstream, start_state, codebook, size);
        if (rc != TCQ_OK) return rc;
        rc = check_matrix(fn, "x", x, ldx, N, size);
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
    if (pre) {
        rc = check_matrix(fn, "pre", pre, ldp, M, size);
        if (rc != TCQ_OK) return rc;
        if (pre == y || pre == residual) {
            set_error("%s: pre must be a buffer of its own", fn);
            return TCQ_EINVAL;
        }
    }
    rc = check_workspace(fn, workspace, workspace_bytes,
                         forward_bytes(dtype, B, M, N, L, k, V, T));
    if (rc != TCQ_OK) return rc;
    const Region rx = region("x", N > 0 ? x : nullptr, B, ldx, N, size);
    const Region ry = region("y", y, B, ldy, M, size), rp = region("pre", pre, B, ldp, M, size);
    const Region rr = region("residual", residual == y ? nullptr : residual, B, ldr, M, size);
    rc = check_apart(fn, ry, rx);
    if (rc == TCQ_OK) rc = check_apart(fn, ry, rr);
    if (rc == TCQ_OK) rc = check_apart(fn, rp, rx);
    if (rc == TCQ_OK) rc = check_apart(fn, rp, ry);
    if (rc == TCQ_OK) rc = check_apart(fn, rp, rr);
    if (rc != TCQ_OK) return rc;
    const CodedMatrix w{bitstream, start_state, codebook, M, N, L, k, V, T};
    const LinearCall c{dtype, act, x, B, ldx, row_scale, bias, residual, ldr, y, ldy, pre, ldp};
    const hipError_t e = launch_linear(w, c, static_cast<char *>(workspace), stream);
    if (e != hipSuccess) return hip_fail(fn, "linear layer launch", e);
    return TCQ_OK;
}

extern "C" int tcq_act_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                            int8_t *codes, int64_t ldq, uint8_t *scale, hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_act_pack";
    int rc = check_pack(fn, dtype, rows, cols);
    if (rc != TCQ_OK) return rc;
    if (rows == 0 || cols == 0) return TCQ_OK;
    rc = check_matrix(fn, "X", X, ldx, cols, size_of(dtype));
    if (rc == TCQ_OK) rc = check_matrix(fn, "codes", codes, ldq, cols, 1);
    if (rc == TCQ_OK) rc = check_matrix(fn, "scale", scale, 0, 0, 1);
    const Region rX = region("X", X, rows, ldx, cols, size_of(dtype));
    const Region rq = region("codes", codes, rows, ldq, cols, 1);
    const Region rs = region("scale", scale, 1, 0, rows * ((cols + 31) / 32), 1);
    if (rc == TCQ_OK) rc = check_apart(fn, rq, rX);
    if (rc == TCQ_OK) rc = check_apart(fn, rs, rX);
    if (rc == TCQ_OK) rc = check_apart(fn, rs, rq);
    if (rc != TCQ_OK) return rc;
    const hipError_t e = launch_act_pack(X, dtype, rows, cols, ldx, codes, ldq, scale, stream);
    if (e != hipSuccess) return hip_fail(fn, "checkpoint launch", e);
    return TCQ_OK;
}

extern "C" int tcq_act_unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale,
                              int64_t rows, int64_t cols, int dtype, void *out, int64_t ldo,
                              hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_act_unpack";
    int rc = check_pack(fn, dtype, rows, cols);
    if (rc != TCQ_OK) return rc;
    if (rows == 0 || cols == 0) return TCQ_OK;
    rc = check_matrix(fn, "codes", codes, ldq, cols, 1);
    if (rc == TCQ_OK) rc = check_matrix(fn, "scale", scale, 0, 0, 1);
    if (rc == TCQ_OK) rc = check_matrix(fn, "out", out, ldo, cols, size_of(dtype));
    const Region ro = region("out", out, rows, ldo, cols, size_of(dtype));
    if (rc == TCQ_OK) rc = check_apart(fn, ro, region("codes", codes, rows, ldq, cols, 1));
    if (rc == TCQ_OK)
        rc = check_apart(fn, ro, region("scale", scale, 1, 0, rows * ((cols + 31) / 32), 1));
    if (rc != TCQ_OK) return rc;
    const hipError_t e =
        launch_act_unpack(codes, ldq, scale, rows, cols, dtype, out, ldo, cols, stream);
    if (e != hipSuccess) return hip_fail(fn, "checkpoint launch", e);
    return TCQ_OK;
}

extern "C" int tcq_decode_linear_backward_workspace_bytes(int dtype, int64_t B, int64_t M,
                                                          int64_t N, int L, int k, int V, int T,
                                                          int dx, int dw, int dbias,
                                                          size_t *bytes) {
    clear_error();
    const char *fn = "tcq_decode_linear_backward_workspace_bytes";
    const int rc = check_layer(fn, dtype, B, M, N, L, k, V, T);
    if (rc != TCQ_OK) return rc;
    if (!bytes) {
        set_error("%s: bytes is NULL", fn);
        return TCQ_EINVAL;
    }
    *bytes = linear_grad_layout(size_of(dtype), B, M, N, dx != 0, dw != 0, dbias != 0, 1).bytes;
    return TCQ_OK;
}

extern "C" int tcq_decode_linear_backward(
    const uint32_t *bitstream, const uint32_t *start_state, const void *codebook, int64_t M,
    int64_t N, int L, int k, int V, int T, int dtype, const void *dy, int64_t B, int64_t lddy,
    const float *row_scale, int act, const int8_t *z_codes, int64_t ldz, const uint8_t *z_scale,
    const int8_t *x_codes, int64_t ldx, const uint8_t *x_scale, void *dx, int64_t lddx, void *dw,
    int64_t lddw, float *dbias, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    const char *fn = "tcq_decode_linear_backward";
    int rc = check_layer(fn, dtype, B, M, N, L, k, V, T);
    if (rc != TCQ_OK) return rc;
    rc = check_act(fn, act);
    if (rc != TCQ_OK) return rc;
    if (!dx && !dw && !dbias) {
        set_error("%s: none of dx, dw and dbias is wanted", fn);
        return TCQ_EINVAL;
    }
    const size_t size = size_of(dtype);
    if (B > 0 && M > 0) {
        rc = check_matrix(fn, "dy", dy, lddy, M, size);
        if (rc == TCQ_OK && act != TCQ_ACT_NONE) {
            rc = check_matrix(fn, "z_codes", z_codes, ldz, M, 1);
            if (rc == TCQ_OK) rc = check_matrix(fn, "z_scale", z_scale, 0, 0, 1);
        }
        if (rc != TCQ_OK) return rc;
    }
    if (dx && B > 0 && N > 0) {
        rc = check_matrix(fn, "dx", dx, lddx, N, size);
        if (rc == TCQ_OK && M > 0) rc = check_coded(fn, bitstream, start_state, codebook, size);
        if (rc != TCQ_OK) return rc;
    }
    if (dw && M > 0 && N > 0) {
        rc = check_matrix(fn, "dw", dw, lddw, N, size);
        if (rc == TCQ_OK && B > 0) {
            rc = check_matrix(fn, "x_codes", x_codes, ldx, N, 1);
            if (rc == TCQ_OK) rc = check_matrix(fn, "x_scale", x_scale, 0, 0, 1);
        }
        if (rc != TCQ_OK) return rc;
    }
    rc = check_workspace(
        fn, workspace, workspace_bytes,
        linear_grad_layout(size, B, M, N, dx != nullptr, dw != nullptr, dbias != nullptr, 1)
            .bytes);
    if (rc != TCQ_OK) return rc;
    const Region rdx = region("dx", N > 0 ? dx : nullptr, B, lddx, N, size);
    const Region rdw = region("dw", N > 0 ? dw : nullptr, M, lddw, N, size);
    const Region rdb = region("dbias", dbias, 1, 0, M, sizeof(float));
    rc = check_apart(fn, rdx, rdw);
    if (rc == TCQ_OK) rc = check_apart(fn, rdx, rdb);
    if (rc == TCQ_OK) rc = check_apart(fn, rdw, rdb);
    if (rc != TCQ_OK) return rc;
    const CodedMatrix w{bitstream, start_state, codebook, M, N, L, k, V, T};
    const LinearGrad c{dtype, act, dy, B, lddy, row_scale, z_codes, ldz, z_scale, x_codes, ldx,
                       x_scale, dx, lddx, dw, lddw, dbias};
    const hipError_t e = launch_linear_grad(w, c, static_cast<char *>(workspace), stream);
    if (e != hipSuccess) return hip_fail(fn, "linear layer gradient launch", e);
    return TCQ_OK;
}
