// 8-bit activation checkpoints: groups of 32 consecutive values of a row share one scale
// byte e, the exponent field of the group's largest magnitude as an fp32 number, and each
// value is held as an int8 code q standing for q 2^(e - 133):
//     q = clamp(round_half_even(x 2^(133 - e)), -127, 127).
// With a power of two as the scale both directions are exact apart from the one rounding
// to an integer, and every code's value is a bf16 number, so a product can read the
// checkpoint without rounding it again.  e = 255 (an infinity or a NaN in the group) makes
// the whole group NaN.
#include <hip/hip_runtime.h>

#include "checkpoint_device.h"
#include "tcq.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

// Eight consecutive values per thread; four neighbouring lanes share a group.
template <typename T, bool SMALL>
__global__ __launch_bounds__(256) void act_pack_kernel(const T *__restrict__ X, Pieces ix,
                                                       int64_t cols, int64_t ldx,
                                                       int8_t *__restrict__ codes, int64_t ldq,
                                                       uint8_t *__restrict__ scale) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < ix.total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        int64_t r;
        uint32_t c;
        split<SMALL>(i, ix.cpr, r, c);
        const int64_t col = static_cast<int64_t>(c) * 8;
        const int left = cols - col < 8 ? static_cast<int>(cols - col) : 8;  // may be <= 0
        float x[8];
        if (left == 8) {
            const Packed<T> e = *reinterpret_cast<const Packed<T> *>(X + r * ldx + col);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = static_cast<float>(e.v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < left ? static_cast<float>(X[r * ldx + col + k]) : 0.0f;
        }
        // magnitudes order like their bit patterns (NaN above infinity)
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t m = __float_as_uint(x[k]) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
        // the group's four lanes: total and the grid are multiples of 4, so they are here
        // together
        uint32_t o = __builtin_amdgcn_update_dpp(0, top, 0xB1, 0xF, 0xF, false);  // lanes 1 0 3 2
        top = top > o ? top : o;
        o = __builtin_amdgcn_update_dpp(0, top, 0x4E, 0xF, 0xF, false);           // lanes 2 3 0 1
        top = top > o ? top : o;
        const int e = static_cast<int>(top >> 23);
        uint32_t word[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float q = __builtin_rintf(__builtin_amdgcn_ldexpf(x[k], 133 - e));
            q = __builtin_amdgcn_fmed3f(q, -127.0f, 127.0f);
            const uint32_t b = e == 255 ? 0u : static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu;
            word[k / 4] |= b << (8 * (k % 4));
        }
        int8_t *q = codes + r * ldq + col;
        if (left == 8) {
            struct __attribute__((packed)) Two { uint32_t a, b; };
            *reinterpret_cast<Two *>(q) = Two{word[0], word[1]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) q[k] = static_cast<int8_t>(word[k / 4] >> (8 * (k % 4)));
        }
        if ((c & 3) == 0) scale[i >> 2] = static_cast<uint8_t>(e);
    }
}

template <typename T, bool SMALL>
__global__ __launch_bounds__(256) void act_unpack_kernel(UnpackArgs a, T *__restrict__ out) {
    act_unpack<T, SMALL>(a, out, blockIdx.x, gridDim.x);
}

unsigned grid_for(int64_t work, int64_t per) {
    int64_t g = (work + per - 1) / per;
    if (g > (1 << 20)) g = 1 << 20;
    return static_cast<unsigned>(g < 1 ? 1 : g);
}

template <typename T>
hipError_t pack(const void *X, int64_t rows, int64_t cols, int64_t ldx, int8_t *codes,
                int64_t ldq, uint8_t *scale, hipStream_t s) {
    const int64_t groups = (cols + kGroup - 1) / kGroup;
    const Pieces ix{static_cast<uint32_t>(groups * 4), rows * groups * 4};
    const auto kern = ix.total < (int64_t{1} << 32) ? act_pack_kernel<T, true>
                                                    : act_pack_kernel<T, false>;
    hipLaunchKernelGGL(kern, dim3(grid_for(ix.total, 256)), dim3(256), 0, s,
                       static_cast<const T *>(X), ix, cols, ldx, codes, ldq, scale);
    return hipGetLastError();
}

template <typename T>
hipError_t unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale, int64_t rows,
                  int64_t cols, void *out, int64_t ldo, int64_t padded, hipStream_t s) {
    const UnpackArgs a = unpack_args<T>(codes, ldq, scale, rows, cols, ldo, padded);
    const auto kern = a.ix.total < (int64_t{1} << 32) ? act_unpack_kernel<T, true>
                                                      : act_unpack_kernel<T, false>;
    hipLaunchKernelGGL(kern, dim3(grid_for(a.ix.total, 256)), dim3(256), 0, s, a,
                       static_cast<T *>(out));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_act_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int8_t *codes, int64_t ldq, uint8_t *scale, hipStream_t s) {
    switch (dtype) {
        case TCQ_F32: return pack<float>(X, rows, cols, ldx, codes, ldq, scale, s);
        case TCQ_F16: return pack<_Float16>(X, rows, cols, ldx, codes, ldq, scale, s);
        default: return pack<__bf16>(X, rows, cols, ldx, codes, ldq, scale, s);
    }
}

hipError_t launch_act_unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale,
                             int64_t rows, int64_t cols, int dtype, void *out, int64_t ldo,
                             int64_t padded, hipStream_t s) {
    switch (dtype) {
        case TCQ_F32: return unpack<float>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
        case TCQ_F16:
            return unpack<_Float16>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
        default: return unpack<__bf16>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
    }
}

}  // namespace tcq
