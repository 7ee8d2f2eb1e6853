// Argument checks that the C ABI's sources share (host code); each returns a status and sets the
// error message.
#pragma once

#include "region.h"
#include "tcq.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

int check_dtype(const char *fn, int dtype) {
    if (dtype != TCQ_F32 && dtype != TCQ_F16 && dtype != TCQ_BF16) {
        set_error("%s: dtype=%d is none of TCQ_F32, TCQ_F16, TCQ_BF16", fn, dtype);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

size_t size_of(int dtype) { return dtype == TCQ_F32 ? 4 : 2; }

int check_format(const char *fn, int format) {
    if (format != TCQ_FP4 && format != TCQ_FP8) {
        set_error("%s: format=%d is none of TCQ_FP4, TCQ_FP8", fn, format);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

// A matrix argument: present, its rows apart and its address a multiple of the value's size.
int check_matrix(const char *fn, const char *name, const void *p, int64_t ld, int64_t cols,
                 size_t size) {
    if (!p) {
        set_error("%s: %s must be non-NULL", fn, name);
        return TCQ_EINVAL;
    }
    if (reinterpret_cast<uintptr_t>(p) % size) {
        set_error("%s: %s at %p is not aligned to its values of %zu bytes", fn, name, p, size);
        return TCQ_EINVAL;
    }
    if (ld < cols) {
        set_error("%s: leading dimension %lld of %s is below its %lld columns", fn,
                  (long long)ld, name, (long long)cols);
        return TCQ_EINVAL;
    }
    return TCQ_OK;
}

int check_apart(const char *fn, const Region &out, const Region &other) {
    if (!out.p || !other.p || !overlap(out, other)) return TCQ_OK;
    set_error("%s: %s and %s overlap", fn, out.name, other.name);
    return TCQ_EINVAL;
}

int check_workspace(const char *fn, const void *workspace, size_t bytes, size_t need) {
    if (need == 0) return TCQ_OK;
    if (!workspace || bytes < need) {
        set_error("%s: workspace of %zu bytes is below the minimum %zu", fn,
                  workspace ? bytes : size_t{0}, need);
        return TCQ_EWORKSPACE;
    }
    return check_workspace_alignment(fn, workspace);
}

}  // namespace
}  // namespace tcq
