// Microscaled quantisation (tcq_mx_pack, tcq_mx_unpack).  A group of 32 consecutive values of a
// row has the scale byte e = max(E - t, 0), E the exponent field of its largest magnitude as an
// fp32 number and t = 2 (E2M1) or 8 (E4M3), and each value the code nearest to x 2^(127 - e),
// ties to even, clamped to 6 or 448.  Multiplying by a power of two is exact, so a code has one
// rounding.  E = 255 (an infinity or a NaN) gives e = 255, which stands for NaN throughout.
//   Both directions are bound by memory: one pass, eight values or 16 bytes of output a thread
// (16384 x 14336 bf16 into 8 bits 129 us, back 126: 5.5 and 5.6 TB/s; 2048 x 2048 fp32 into 4 bits
// 4.2, back 4.9, about twice a launch).
#include <hip/hip_runtime.h>

#include "checkpoint_device.h"
#include "mx_unpack_device.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

struct MxPackArgs {
    const void *x;
    int64_t cols, ldx;
    Pieces ix;          // pieces of eight values, whole groups
    uint8_t *codes;     // rows of ldq bytes, or NULL
    int64_t ldq;
    uint8_t *scale;     // rows x groups, or NULL
    __bf16 *values;     // the values the codes stand for, rows of ldv, or NULL
    int64_t ldv;
    MxOrder order;      // codes NULL: not wanted
    uint32_t groups;    // of a row (pieces go on to whole pairs where an order is wanted)
};

// Eight consecutive values per thread; four neighbouring lanes share a group.
template <typename T, int FMT, bool SMALL>
__global__ __launch_bounds__(256) void mx_pack_kernel(MxPackArgs a) {
    const T *X = static_cast<const T *>(a.x);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < a.ix.total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        int64_t r;
        uint32_t c;
        split<SMALL>(i, a.ix.cpr, r, c);
        const int64_t col = static_cast<int64_t>(c) * 8;
        const int left = a.cols - col < 8 ? static_cast<int>(a.cols - col) : 8;  // may be <= 0
        float x[8];
        if (left == 8) {
            const Packed<T> p = *reinterpret_cast<const Packed<T> *>(X + r * a.ldx + col);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = static_cast<float>(p.v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < left ? static_cast<float>(X[r * a.ldx + col + k]) : 0.0f;
        }
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t m = __float_as_uint(x[k]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
        // (total and the grid are multiples of 4: a group's lanes are here together)
        const int e = mx::scale_byte<FMT>(mx::group_top(top));
        uint32_t w[2];
        mx::encode8<FMT>(x, e, w);
        if (a.order.codes) {
            // pair, tile of 16 rows, group of the lane's two, (half,) lane; 16 bytes each
            const uint32_t grp = c >> 2, part = c & 3, pair = grp >> 3, k = grp & 1;
            const uint32_t lane = (grp & 7) / 2 * 16 + (static_cast<uint32_t>(r) & 15);
            const int64_t at = static_cast<int64_t>(pair) * a.order.nbt + (r >> 4);
            if constexpr (FMT == TCQ_FP4)
                reinterpret_cast<uint32_t *>(a.order.codes)[((at * 2 + k) * 64 + lane) * 4 + part] =
                    w[0];
            else
                reinterpret_cast<uint2 *>(
                    a.order.codes)[(((at * 2 + k) * 2 + part / 2) * 64 + lane) * 2 + part % 2] =
                    make_uint2(w[0], w[1]);
            if (part == 0) a.order.scale[(at * 64 + lane) * 2 + k] = static_cast<uint8_t>(e);
            if (grp >= a.groups) continue;
        }
        if (a.codes) {
            uint8_t *q = a.codes + r * a.ldq + static_cast<int64_t>(c) * mx::bytes<FMT>(8);
            if constexpr (FMT == TCQ_FP4)
                *reinterpret_cast<uint32_t *>(q) = w[0];
            else
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        }
        if (a.scale && (c & 3) == 0) a.scale[r * a.groups + (c >> 2)] = static_cast<uint8_t>(e);
        if (a.values) {
            const float s = mx::scale_of(e);
            uint32_t v[4];
            mx::decode_word_bf16<FMT>(w[0], s, v);
            if constexpr (FMT == TCQ_FP8) mx::decode_word_bf16<FMT>(w[1], s, v + 2);
            *reinterpret_cast<uint4 *>(a.values + r * a.ldv + col) =
                make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

template <typename T, int FMT, bool SMALL>
__global__ __launch_bounds__(256) void mx_unpack_kernel(MxUnpackArgs a, T *__restrict__ out) {
    mx_unpack<T, FMT, SMALL>(a, out, blockIdx.x, gridDim.x);
}

unsigned grid_for(int64_t work, int64_t per) {
    int64_t g = (work + per - 1) / per;
    if (g > (1 << 20)) g = 1 << 20;
    return static_cast<unsigned>(g < 1 ? 1 : g);
}

template <typename T, int FMT>
hipError_t pack(MxPackArgs a, hipStream_t s) {
    const auto kern = a.ix.total < (int64_t{1} << 32) ? mx_pack_kernel<T, FMT, true>
                                                      : mx_pack_kernel<T, FMT, false>;
    hipLaunchKernelGGL(kern, dim3(grid_for(a.ix.total, 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename T, int FMT>
hipError_t unpack(const MxMatrix &m, int64_t rows, int64_t cols, void *out, int64_t ldo,
                  int64_t padded, hipStream_t s) {
    const MxUnpackArgs a = mx_unpack_args<T>(m, rows, cols, ldo, padded);
    const auto kern = a.ix.total < (int64_t{1} << 32) ? mx_unpack_kernel<T, FMT, true>
                                                      : mx_unpack_kernel<T, FMT, false>;
    hipLaunchKernelGGL(kern, dim3(grid_for(a.ix.total, 256)), dim3(256), 0, s, a,
                       static_cast<T *>(out));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                          int format, uint8_t *codes, int64_t ldq, uint8_t *scale,
                          uint16_t *values, int64_t ldv, const MxOrder *order, hipStream_t s) {
    const int64_t groups = (cols + mx::kGroup - 1) / mx::kGroup;
    const int64_t cpr = (order ? (groups + 7) / 8 * 8 : groups) * 4;
    const MxPackArgs a{X, cols, ldx, {static_cast<uint32_t>(cpr), rows * cpr}, codes, ldq, scale,
                       reinterpret_cast<__bf16 *>(values), ldv,
                       order ? *order : MxOrder{nullptr, nullptr, 0},
                       static_cast<uint32_t>(groups)};
    const bool fp4 = format == TCQ_FP4;
    switch (dtype) {
        case TCQ_F32: return fp4 ? pack<float, TCQ_FP4>(a, s) : pack<float, TCQ_FP8>(a, s);
        case TCQ_F16: return fp4 ? pack<_Float16, TCQ_FP4>(a, s) : pack<_Float16, TCQ_FP8>(a, s);
        default: return fp4 ? pack<__bf16, TCQ_FP4>(a, s) : pack<__bf16, TCQ_FP8>(a, s);
    }
}

hipError_t launch_mx_unpack(const MxMatrix &m, int64_t rows, int64_t cols, int dtype, void *out,
                            int64_t ldo, int64_t padded, hipStream_t s) {
    const bool fp4 = m.format == TCQ_FP4;
#define TCQ_UNPACK(T)                                                                     \
    (fp4 ? unpack<T, TCQ_FP4>(m, rows, cols, out, ldo, padded, s)               \
         : unpack<T, TCQ_FP8>(m, rows, cols, out, ldo, padded, s))
    switch (dtype) {
        case TCQ_F32: return TCQ_UNPACK(float);
        case TCQ_F16: return TCQ_UNPACK(_Float16);
        default: return TCQ_UNPACK(__bf16);
    }
#undef TCQ_UNPACK
}

}  // namespace tcq
