// What becomes of a product's sums: the layer's outputs, plain outputs, or one split's share
// (device code), the kernel that joins shares, and the sum of slabs.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_device.h"
#include "linear_device.h"

namespace tcq {
namespace {

using gemm::f32x4;

template <typename T>
__device__ __forceinline__ void store4(T *p, int64_t j, int64_t J, bool vec, f32x4 v) {
    struct alignas(4 * sizeof(T)) Four { T v[4]; } o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.v[e] = static_cast<T>(v[e]);
    if (vec && j + 4 <= J) {
        *reinterpret_cast<Four *>(p) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < J) p[e] = o.v[e];
    }
}

template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p, int64_t j, int64_t J, bool vec) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (vec && j + 4 <= J) {
        struct alignas(4 * sizeof(T)) Four { T v[4]; };
        const Four o = *reinterpret_cast<const Four *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(o.v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < J) v[e] = static_cast<float>(p[e]);
    }
    return v;
}

// y = act(scale s + bias) + residual, z = scale s + bias, in fp32, rounded once each.
template <typename T>
struct LayerEpilogue {
    const float *scale;
    const float *bias;
    const T *res;
    T *y;
    T *pre;
    int64_t ldr, ldy, ldp;
    int64_t I, J;
    int act;
    int vec_y, vec_r, vec_p;  // four consecutive values are aligned

    struct Column {
        int64_t j;
        f32x4 a, b;
        __device__ __forceinline__ Column(const LayerEpilogue &e, int64_t j_) : j(j_) {
            a = f32x4{1.f, 1.f, 1.f, 1.f};
            b = f32x4{0.f, 0.f, 0.f, 0.f};
            if (e.scale && j < e.J) a = load4(e.scale + j, j, e.J, false);
            if (e.bias && j < e.J) b = load4(e.bias + j, j, e.J, false);
        }
    };
    __device__ __forceinline__ void put(const Column &c, int64_t i, f32x4 s) const {
        if (i >= I || c.j >= J) return;
        f32x4 z, o;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = __builtin_fmaf(c.a[e], s[e], c.b[e]);
        if (pre) store4(pre + i * ldp + c.j, c.j, J, vec_p, z);
        with_act(act, [&](auto a) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = act_value<decltype(a)::value, sizeof(T) == 4>(z[e]);
        });
        if (res) {
            const f32x4 r = load4(res + i * ldr + c.j, c.j, J, vec_r);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += r[e];
        }
        store4(y + i * ldy + c.j, c.j, J, vec_y, o);
    }
    __device__ __forceinline__ void put_one(int64_t i, int64_t j, float s) const {
        if (i >= I || j >= J) return;
        const float z = __builtin_fmaf(scale ? scale[j] : 1.0f, s, bias ? bias[j] : 0.0f);
        if (pre) pre[i * ldp + j] = static_cast<T>(z);
        float o = 0.0f;
        with_act(act, [&](auto a) { o = act_value<decltype(a)::value, sizeof(T) == 4>(z); });
        if (res) o += static_cast<float>(res[i * ldr + j]);
        y[i * ldy + j] = static_cast<T>(o);
    }
};

// The sums times 2^*exponent (NULL: 1), rounded once.
template <typename T>
struct PlainEpilogue {
    T *y;
    int64_t ldy, I, J;
    int vec_y;
    const int *exponent;
    struct Column {
        int64_t j;
        int e;
        __device__ __forceinline__ Column(const PlainEpilogue &p, int64_t j_)
            : j(j_), e(p.exponent ? *p.exponent : 0) {}
    };
    __device__ __forceinline__ void put(const Column &c, int64_t i, f32x4 s) const {
        if (i >= I || c.j >= J) return;
        if constexpr (gemm::kLowShift<T> != 0) {
#pragma unroll
            for (int v = 0; v < 4; ++v) s[v] = __builtin_amdgcn_ldexpf(s[v], c.e);
        }
        store4(y + i * ldy + c.j, c.j, J, vec_y, s);
    }
};

// One split's share of the sums over k, in fp32: part[split][i][j], rows of ld values.
struct PartEpilogue {
    float *part;
    int64_t ld, I, J;
    struct Column {
        int64_t j;
        __device__ __forceinline__ Column(const PartEpilogue &, int64_t j_) : j(j_) {}
    };
    __device__ __forceinline__ void put(const Column &c, int64_t i, f32x4 s) const {
        if (i < I && c.j < J) *reinterpret_cast<f32x4 *>(part + i * ld + c.j) = s;
    }
};

// The splits' shares added in order, four values per thread, and handed to the epilogue.
template <typename Epi>
__global__ __launch_bounds__(256) void split_sum_kernel(const float *__restrict__ part, int splits,
                                                        int64_t I, int64_t ld, Epi epi) {
    const int64_t quads = ld / 4;
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (q >= I * quads) return;
    const int64_t i = q / quads, j = (q - i * quads) * 4;
    const float *p = part + i * ld + j;
    f32x4 s = *reinterpret_cast<const f32x4 *>(p);
    for (int v = 1; v < splits; ++v) s += *reinterpret_cast<const f32x4 *>(p + v * I * ld);
    const typename Epi::Column col(epi, j);
    epi.put(col, i, s);
}

// sum[c] = part[0][c] + part[1][c] + ...: each of four waves adds a run of slabs in order, then
// the four sums in order; 64 columns per workgroup.
__device__ __forceinline__ void slab_sum(const float *__restrict__ part, int64_t slabs, int64_t M,
                                         float *__restrict__ sum, uint32_t block) {
    __shared__ float red[4][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = static_cast<int64_t>(block) * 64 + lane;
    const int64_t i0 = w * slabs / 4, i1 = (w + 1) * slabs / 4;
    float s = 0.0f;
    if (c < M) {
#pragma unroll 8
        for (int64_t i = i0; i < i1; ++i) s += part[i * M + c];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < M) sum[c] = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
}

template <typename T>
bool four_aligned(const T *p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T))) == 0 && ld % 4 == 0;
}

}  // namespace
}  // namespace tcq
