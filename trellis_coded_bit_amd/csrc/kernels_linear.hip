// The coded linear layer: y = act(row_scale (x W_hat^T) + bias) + residual for a batch of
// rows x, with the trellis-coded matrix W_hat decoded inside the call, and its gradients.
//
// The matrix is decoded once into the workspace, in the layer's type, and multiplied on the
// matrix cores (gemm_device.h); for few rows it is decoded inside the product.  With the table
// in the layer's own type a decoded weight is a table entry copied bit for bit, so every
// product is exact and the sums are fp32: the outputs' own rounding is the only one to 16 bits.  The backward pass holds the incoming
// gradient times the activation's slope and the row scale in two terms of a 16-bit type, since
// its products read it through the matrix cores: rounded to one term, dx and dw were off by 1.4
// times their own rounding, and in fp16 the row scale (about 1 / sqrt N) pushed small gradients
// among the subnormals (11 % off at a gradient of 1e-5).  It costs a second pass over k
// (4096 x 4096 x 4096: 220-255 us a product, 113-119 with one term).
#include <hip/hip_runtime.h>

#include "checkpoint_device.h"
#include "decode_device.h"
#include "gemm_device.h"
#include "linear_device.h"
#include "tcq.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

using gemm::f32x4;
using gemm::Operand;

// ---------------------------------------------------------------- decode into memory

struct DecodeArgs {
    const uint32_t *bits;
    const uint32_t *s0;
    const void *table;
    int64_t M, N, ld;  // out is M x ld, ld >= N a multiple of 8; columns past N are zeros
    int L, kv, V, T, nwords;
};

// Any trellis: a thread decodes eight consecutive columns, each on its own.  Step t's state
// is the L-bit window of s_0 || b_1 || ... that ends with b_t, inside the word that holds
// the chunk's last bit and the word before it (s_0 for the first word).
template <typename T>
__global__ __launch_bounds__(256) void decode_matrix_kernel(DecodeArgs a, T *__restrict__ out) {
    const int64_t cpr = a.ld / 8;
    const int64_t chunks = a.M * cpr;
    const int64_t bpr = a.N / a.T;
    const T *table = static_cast<const T *>(a.table);
    const uint32_t mask = (1u << a.L) - 1u;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < chunks;
         q += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = q / cpr;
        const int64_t c0 = (q - row * cpr) * 8;
        struct alignas(8 * sizeof(T)) Eight { T v[8]; } o;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + e;
            T w = static_cast<T>(0.0f);
            if (c < a.N) {
                const int64_t blk = row * bpr + c / a.T;
                const int i = static_cast<int>(c % a.T);
                const int end = (i / a.V + 1) * a.kv;  // stream bits up to the chunk's end
                const int j = (end - 1) >> 5;
                const uint32_t *wb = a.bits + blk * a.nwords;
                const uint32_t hi = j ? wb[j - 1] : a.s0[blk];
                const uint32_t st =
                    __builtin_amdgcn_alignbit(hi, wb[j], 32 * (j + 1) - end) & mask;
                w = table[static_cast<int64_t>(st) * a.V + i % a.V];
            }
            o.v[e] = w;
        }
        *reinterpret_cast<Eight *>(out + row * a.ld + c0) = o;
    }
}

// Blocks of whole chunks (T a multiple of 8): eight columns per thread and turn, decoded
// from the table in LDS.  The matrix is dense then (ld = N), so chunk g's values are out's
// values 8 g .. 8 g + 7 and its block is g / (T / 8).  A table of more than 128 KiB goes
// through LDS in parts: every pass ORs in the steps whose state lies in its part, the others
// read a row of zeros after the part, so the values' bits arrive unchanged.
struct ChunkArgs {
    const uint32_t *bits;
    const uint32_t *s0;
    const char *table;
    uint32_t chunks;         // of the matrix
    uint32_t chunks_per_wg;
    int rows;                // chunks per thread and turn
    uint32_t cpb;            // chunks per block
    int cpb_log2;            // log2(cpb), or -1
    int L, nwords;
    int part_log2;           // log2(states per part)
    int parts;
    int vec;                 // the table is 16-byte aligned
};

constexpr int kChunkThreads = 1024;
constexpr int kPartBytes = 128 << 10;

// Chunks a thread holds at a time.  With several parts each keeps its values over the
// passes (14336 x 4096, V = 2, 16 bits: 41-42 us with 7 to 14, 44 with 5); with one, two keep
// the stores flowing (4096 x 4096, 16 bits: 12.9 us with 2 or 4, 14.1 with 8).
template <typename T, bool ONE>
constexpr int chunk_rows() {
    return ONE ? 2 : (sizeof(T) == 4 ? 8 : 14);
}

template <typename T, int KV, int V, bool ONE>
__global__ __launch_bounds__(kChunkThreads) void decode_chunks_kernel(ChunkArgs a,
                                                                      T *__restrict__ out) {
    using C = Chunk<KV, V>;
    constexpr int RT = chunk_rows<T, ONE>();
    constexpr int kRowBytes = V * static_cast<int>(sizeof(T));
    constexpr int kLog = kRowBytes == 2 ? 1 : (kRowBytes == 4 ? 2 : (kRowBytes == 8 ? 3 : 4));
    constexpr int kWords = 8 * static_cast<int>(sizeof(T)) / 4;  // 32-bit words of a chunk
    extern __shared__ __align__(16) char tab[];
    const int tid = threadIdx.x;
    const int part_bytes = 1 << (a.part_log2 + kLog);
    const uint32_t dummy = static_cast<uint32_t>(part_bytes);
    const uint32_t begin = blockIdx.x * a.chunks_per_wg;
    const uint32_t end = begin + a.chunks_per_wg < a.chunks ? begin + a.chunks_per_wg : a.chunks;
    auto copy = [&](int p) {
        table_to_lds<kChunkThreads>(tab, a.table + static_cast<int64_t>(p) * part_bytes,
                                    part_bytes, sizeof(T), a.vec, tid);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (!ONE) {
            if (tid < 4) reinterpret_cast<uint32_t *>(tab + part_bytes)[tid] = 0u;
            __syncthreads();
        }
    };
    // the values of chunk words n whose states lie in the part that starts at `base`
    auto decode = [&](const uint32_t (&n)[C::NW], uint32_t base, uint32_t (&val)[kWords]) {
#pragma unroll
        for (int t = 0; t < C::kSteps; ++t) {
            uint32_t off = chunk_state<KV, V>(n, t, a.L) << kLog;
            if (!ONE) {
                off -= base;  // wraps below the part
                off = off < dummy ? off : dummy;
            }
            const char *row = tab + off;
            if constexpr (kRowBytes == 2) {
                const uint32_t v = *reinterpret_cast<const uint16_t *>(row);
                val[t / 2] |= v << (16 * (t % 2));
            } else {
#pragma unroll
                for (int j = 0; j < kRowBytes / 4; ++j)
                    val[t * (kRowBytes / 4) + j] |= reinterpret_cast<const uint32_t *>(row)[j];
            }
        }
    };
    if (ONE) copy(0);
    int first = 0;  // the tile's first part: the one the previous tile ended with
    for (uint32_t t0 = begin; t0 < end; t0 += kChunkThreads * a.rows) {
        uint32_t n[RT][C::NW];
        uint32_t val[RT][kWords];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (i < a.rows) {
                uint32_t g = t0 + i * kChunkThreads + tid;
                g = g < end ? g : begin;  // (decoded again and not stored)
                const uint32_t blk = a.cpb_log2 >= 0 ? g >> a.cpb_log2 : g / a.cpb;
                const int q = static_cast<int>(g - blk * a.cpb);
                uint32_t w[C::NW + 1];
                chunk_words<KV, V>(a.bits + static_cast<int64_t>(blk) * a.nwords, a.s0 + blk, q,
                                   w);
                chunk_align<KV, V>(w, q, n[i]);
            } else {
#pragma unroll
                for (int j = 0; j < C::NW; ++j) n[i][j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < kWords; ++j) val[i][j] = 0u;
        }
        const int parts = ONE ? 1 : a.parts;
        for (int v = 0; v < parts; ++v) {
            const int p = first == 0 ? v : parts - 1 - v;
            if (!ONE && (v > 0 || t0 == begin)) {
                __syncthreads();  // the previous part is done with
                copy(p);
            }
            const uint32_t base = static_cast<uint32_t>(p) * dummy;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                if (i < a.rows) {
                    if constexpr (!ONE) {
                        // (the states are extracted again for every part, one instruction
                        // each, rather than kept in registers)
#pragma unroll
                        for (int j = 0; j < C::NW; ++j) asm volatile("" : "+v"(n[i][j]));
                    }
                    decode(n[i], base, val[i]);
                    if constexpr (!ONE) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        first = first == 0 ? parts - 1 : 0;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const uint32_t g = t0 + i * kChunkThreads + tid;
            if (i < a.rows && g < end) {
                uint4 *o = reinterpret_cast<uint4 *>(out + static_cast<int64_t>(g) * 8);
#pragma unroll
                for (int j = 0; j < kWords; j += 4)
                    o[j / 4] = make_uint4(val[i][j], val[i][j + 1], val[i][j + 2], val[i][j + 3]);
            }
        }
    }
}

// Rows of x into a padded, aligned copy: out is B x ld, columns past N zeros.
template <typename T>
__global__ __launch_bounds__(256) void stage_kernel(const T *__restrict__ x, int64_t B, int64_t N,
                                                    int64_t ldx, T *__restrict__ out,
                                                    int64_t ld) {
    const int64_t total = B * ld;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total;
         q += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = q / ld, c = q - r * ld;
        out[q] = c < N ? x[r * ldx + c] : static_cast<T>(0.0f);
    }
}

// ---------------------------------------------------------------- epilogues

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

// ---------------------------------------------------------------- products

template <typename T, bool AKM, bool BKM, int TI, int TJ, int WI, int WJ, int NB, int TERMS,
          typename Epi>
__global__ __launch_bounds__(WI *WJ * 64) void gemm_kernel(Operand<T> A, Operand<T> B,
                                                           int steps, int steps_per_split,
                                                           Epi epi, uint32_t ni, uint32_t nj) {
    static_assert(NB == 2 || NB == 4 || NB == gemm::kRing, "stages");
    __shared__ __align__(16) char a0[TI * gemm::kStepBytes];
    __shared__ __align__(16) char a1[TI * gemm::kStepBytes];
    __shared__ __align__(16) char b0[TJ * gemm::kStepBytes];
    __shared__ __align__(16) char b1[TJ * gemm::kStepBytes];
    gemm::Stages<NB> st;
    st.a[0] = a0;
    if constexpr (NB == gemm::kRing) {
        static_assert(TI == TJ, "pieces of one size");
        __shared__ __align__(16) char a2[TI * gemm::kStepBytes];
        st.p[0] = a0;
        st.p[1] = b0;
        st.p[2] = a1;
        st.p[3] = b1;
        st.p[4] = a2;
    } else {
        st.a[1] = a1;
        st.b[0] = b0;
        st.b[1] = b1;
    }
    if constexpr (NB == 4) {
        __shared__ __align__(16) char a2[TI * gemm::kStepBytes];
        __shared__ __align__(16) char a3[TI * gemm::kStepBytes];
        __shared__ __align__(16) char b2[TJ * gemm::kStepBytes];
        __shared__ __align__(16) char b3[TJ * gemm::kStepBytes];
        st.a[2] = a2;
        st.a[3] = a3;
        st.b[2] = b2;
        st.b[3] = b3;
    }
    uint32_t ti, tj;
    gemm::tile_of(blockIdx.x, ni, nj, ti, tj);
    const int s0 = blockIdx.y * steps_per_split;
    const int s1 = s0 + steps_per_split < steps ? s0 + steps_per_split : steps;
    if constexpr (__is_same(Epi, PartEpilogue))
        epi.part += static_cast<int64_t>(blockIdx.y) * epi.I * epi.ld;
    const int64_t i0 = static_cast<int64_t>(ti) * TI, j0 = static_cast<int64_t>(tj) * TJ;
    if constexpr (sizeof(T) == 4)
        gemm::gemm_tile_f32<AKM, BKM, TI, TJ, WI, WJ>(A, B, i0, j0, s0, s1, st, epi);
    else
        gemm::gemm_tile<T, AKM, BKM, TI, TJ, WI, WJ, NB, TERMS>(A, B, i0, j0, s0, s1, st, epi);
}

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

template <typename T, bool AKM, bool BKM, int TI, int TJ, int WI, int WJ, int NB, int TERMS,
          typename Epi>
hipError_t launch_tiles(const Operand<T> &A, const Operand<T> &B, const GemmPlan &pl,
                        const Epi &epi, hipStream_t s) {
    const uint32_t ni = static_cast<uint32_t>((A.rows + TI - 1) / TI);
    const uint32_t nj = static_cast<uint32_t>((B.rows + TJ - 1) / TJ);
    hipLaunchKernelGGL((gemm_kernel<T, AKM, BKM, TI, TJ, WI, WJ, NB, TERMS, Epi>),
                       dim3(ni * nj, static_cast<unsigned>(pl.splits)), dim3(WI * WJ * 64), 0, s,
                       A, B, pl.steps, pl.steps_per_split, epi, ni, nj);
    return hipGetLastError();
}

template <typename T, bool AKM, bool BKM, int TERMS, typename Epi>
hipError_t launch_gemm(const Operand<T> &A, const Operand<T> &B, const GemmPlan &pl,
                       const Epi &epi, char *part, hipStream_t s) {
    if (A.rows <= 0 || B.rows <= 0) return hipSuccess;
    if (pl.splits > 1) {
        const PartEpilogue pe{reinterpret_cast<float *>(part), pl.part_ld, A.rows, B.rows};
        // (256 x 256 tiles are not split)
        const hipError_t e =
            pl.tile == kTile128
                ? launch_tiles<T, AKM, BKM, 128, 128, 2, 2, sizeof(T) == 2 ? 4 : 2, TERMS>(
                      A, B, pl, pe, s)
                : launch_tiles<T, AKM, BKM, 64, 128, 1, 4, 2, TERMS>(A, B, pl, pe, s);
        if (e != hipSuccess) return e;
        const int64_t quads = A.rows * (pl.part_ld / 4);
        hipLaunchKernelGGL(split_sum_kernel<Epi>, dim3(static_cast<unsigned>((quads + 255) / 256)),
                           dim3(256), 0, s, pe.part, pl.splits, A.rows, pl.part_ld, epi);
        return hipGetLastError();
    }
    if constexpr (sizeof(T) == 2) {
        if (pl.tile == kTile256)
            return launch_tiles<T, AKM, BKM, 256, 256, 2, 4, gemm::kRing, TERMS>(A, B, pl, epi,
                                                                                 s);
    }
    if (pl.tile == kTile128)
        return launch_tiles<T, AKM, BKM, 128, 128, 2, 2, sizeof(T) == 2 ? 4 : 2, TERMS>(A, B, pl,
                                                                                        epi, s);
    return launch_tiles<T, AKM, BKM, 64, 128, 1, 4, 2, TERMS>(A, B, pl, epi, s);
}

// ---------------------------------------------------------------- few rows of x

// y for a few rows of x (at most 16 BT) with the matrix decoded inside the product: nothing
// but the streams, x and y moves through memory.  A workgroup of 16 waves takes 16 rows of
// the matrix at a time; the waves split its columns into units of 128.
//   Lane (row l16, group g) reads the K words of columns 32 g .. 32 g + 31 of a unit and the
// word before them: the vector memory unit takes about four clocks per cache line of an
// instruction, and a read per chunk (two or three words of 16 rows each) had bounded the
// kernel (one row, 4096 x 14336 at k = 3: 45 us per call, now 18).  Its four chunks are
// aligned with constant shifts and exchanged between the lane groups, so that in step s lane (l16, g)
// holds columns 32 s + 8 g .. + 7, its piece of the matrix instruction's first operand,
// decodes it from the table in LDS and multiplies with 16 rows of x.  Up to 16 rows of x
// are read as they are (any alignment); more are first laid out by pack_rows_kernel in the
// order the steps read them, one contiguous KiB per instruction, since reads of 16 rows cost
// 16 cache lines each.  The waves' sums meet in LDS and are added in wave order.
//   A table of more than 128 KiB goes through LDS in parts; TR tiles' units are then held
// decoded in registers while the parts pass (a step whose state lies elsewhere reads a row
// of zeros), so that each weight is multiplied once, whatever x holds.
constexpr int kSmallWaves = 16;

struct SmallArgs {
    const uint32_t *bits;
    const uint32_t *s0;
    const char *table;
    const void *x;
    int64_t B, ldx;
    int64_t M;
    uint32_t runs;     // per row, N / 32
    uint32_t rpb;      // runs per block
    int rpb_log2;
    uint32_t bpr;      // blocks per row
    int L;
    int part_bytes;    // a power of two
    int parts;
    int red;           // byte offset of the waves' sums in LDS
    int vec;
};

template <typename T, int BT, bool ONE>
struct SmallShape {
    // tiles held at a time, and units held per tile (by the registers: 1024 threads have 128
    // each, and with a table of several parts the instances of fp32 above 32 rows (and one of
    // 17 to 32) and of 16 bits up to 32 rows spill 2 to 18 of them, 27 of all 130)
    static constexpr int TR = ONE || sizeof(T) == 4 || BT > 2 ? 1 : 2;
    static constexpr int UN = ONE || (sizeof(T) == 4 && BT > 4) ? 1 : 2;
    // steps ahead that x is asked for (one less than a divisor of 4; by the registers)
    static constexpr int kAhead =
        BT == 1 ? 3 : (BT * static_cast<int>(sizeof(T)) <= 8 ? 1 : 0);
    // tiles and batch tiles whose sums meet at a time (16 KiB each, beside the table)
    static constexpr int kSumsR = ONE ? TR : 1;
    static constexpr int kSums = ONE && BT > 1 ? 2 : 1;
};

// x as small_kernel's steps read it: the 16-byte piece p of lane l for step s and batch tile t
// is piece ((s BT + t) P + p) 64 + l, where P is the pieces of 8 values.  Rows past B are
// zeros.
template <typename T, int BT>
__global__ __launch_bounds__(256) void pack_rows_kernel(const T *__restrict__ x, int64_t B,
                                                        int64_t ldx, int64_t pieces,
                                                        uint4 *__restrict__ out) {
    constexpr int P = static_cast<int>(sizeof(T)) / 2;
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    struct __attribute__((packed, aligned(2))) Raw { uint32_t w[4]; };
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < pieces;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int l = static_cast<int>(i & 63);
        const int64_t q = i >> 6;
        const int p = static_cast<int>(q % P);
        const int t = static_cast<int>(q / P % BT);
        const int64_t s = q / (P * BT);
        const int64_t b = t * 16 + (l & 15);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (b < B) {
            const Raw r = *reinterpret_cast<const Raw *>(x + b * ldx + s * 32 + (l >> 4) * 8 +
                                                         p * kPer);
            v = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
        out[i] = v;
    }
}

template <typename T, int KV, int V, int BT, bool ONE>
__global__ __launch_bounds__(kSmallWaves * 64) void small_kernel(SmallArgs a,
                                                                 LayerEpilogue<T> epi) {
    using C = Chunk<KV, V>;
    using Tr = gemm::Traits<T>;
    constexpr int K = KV / V;
    using Sh = SmallShape<T, BT, ONE>;
    constexpr int TR = Sh::TR, UN = Sh::UN, kSums = Sh::kSums, kSumsR = Sh::kSumsR;
    constexpr bool kPacked = BT > 1;
    constexpr int kRow = V * static_cast<int>(sizeof(T));  // bytes of a table row
    constexpr int kLog = kRow == 2 ? 1 : (kRow == 4 ? 2 : (kRow == 8 ? 3 : 4));
    constexpr int kWords = 2 * static_cast<int>(sizeof(T));  // 32-bit words of a chunk
    constexpr int kThreads = kSmallWaves * 64;
    struct __attribute__((packed, aligned(2))) Piece { uint32_t w[kWords]; };
    struct __attribute__((packed, aligned(4))) RunWords { uint32_t w[K]; };
    extern __shared__ __align__(16) char tab[];
    float *red = reinterpret_cast<float *>(tab + a.red);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t units = (a.runs + 3) / 4;
    const uint32_t u_begin = wave * units / kSmallWaves;
    const uint32_t u_end = (wave + 1) * units / kSmallWaves;
    // every wave takes the same number of turns: they meet at the table's parts
    const uint32_t most = (units + kSmallWaves - 1) / kSmallWaves;
    const uint32_t dummy = static_cast<uint32_t>(a.part_bytes);
    // rows past B read the last one; their sums are not stored
    const T *xrow = static_cast<const T *>(a.x) + (l16 < a.B ? l16 : a.B - 1) * a.ldx + g * 8;
    const uint4 *xp = static_cast<const uint4 *>(a.x) + lane;
    // step s's piece of batch tile t
    auto read_x = [&](uint32_t s, int t) {
        Piece v;
        if constexpr (kPacked) {
#pragma unroll
            for (int p = 0; p < kWords / 4; ++p) {
                const uint4 q = xp[((s * BT + t) * (kWords / 4) + p) * 64];
                v.w[4 * p] = q.x;
                v.w[4 * p + 1] = q.y;
                v.w[4 * p + 2] = q.z;
                v.w[4 * p + 3] = q.w;
            }
        } else {
            v = *reinterpret_cast<const Piece *>(xrow + s * 32);
        }
        return v;
    };
    auto copy = [&](int p) {
        table_to_lds<kThreads>(tab, a.table + static_cast<int64_t>(p) * a.part_bytes,
                               a.part_bytes, sizeof(T), a.vec, tid);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (!ONE) {
            if (tid < 4) reinterpret_cast<uint32_t *>(tab + a.part_bytes)[tid] = 0u;
            __syncthreads();
        }
    };
    // words of unit u of a matrix row, this lane's run of it
    auto request = [&](const uint32_t *rbits, const uint32_t *rs0, uint32_t u,
                       uint32_t (&w)[K + 1]) {
        uint32_t run = u * 4 + g;
        run = run < a.runs ? run : a.runs - 1;  // (decoded and not multiplied)
        const uint32_t blk = a.rpb_log2 >= 0 ? run >> a.rpb_log2 : run / a.rpb;
        const uint32_t *p = rbits + run * K;
        const uint32_t *before = run == blk * a.rpb ? rs0 + blk : p - 1;
        w[0] = *before;
        const RunWords r = *reinterpret_cast<const RunWords *>(p);
#pragma unroll
        for (int i = 0; i < K; ++i) w[i + 1] = r.w[i];
    };
    // the unit's four chunks as the steps need them
    auto align = [&](const uint32_t (&w)[K + 1], uint32_t (&n)[4][C::NW]) {
#pragma unroll
        for (int s = 0; s < 4; ++s) run_align<KV, V>(w, s, n[s]);
#pragma unroll
        for (int i = 0; i < C::NW; ++i) transpose4(n[0][i], n[1][i], n[2][i], n[3][i]);
    };
    auto decode = [&](const uint32_t (&n)[C::NW], uint32_t base, uint32_t (&val)[kWords]) {
#pragma unroll
        for (int t = 0; t < C::kSteps; ++t) {
            uint32_t off = chunk_state<KV, V>(n, t, a.L) << kLog;
            if (!ONE) {
                off -= base;  // wraps below the part
                off = off < dummy ? off : dummy;
            }
            const char *row = tab + off;
            if constexpr (kRow == 2) {
                const uint32_t v = *reinterpret_cast<const uint16_t *>(row);
                val[t / 2] |= v << (16 * (t % 2));
            } else {
#pragma unroll
                for (int j = 0; j < kRow / 4; ++j)
                    val[t * (kRow / 4) + j] |= reinterpret_cast<const uint32_t *>(row)[j];
            }
        }
    };
    auto multiply = [&](const uint32_t (&val)[kWords], const Piece &x, f32x4 acc) {
        if constexpr (sizeof(T) == 2) {
            struct Four { uint32_t w[4]; };
            const Four v{{val[0], val[1], val[2], val[3]}};
            const Four xx{{x.w[0], x.w[1], x.w[2], x.w[3]}};
            return Tr::mma(__builtin_bit_cast(gemm::s16x8, v),
                           __builtin_bit_cast(gemm::s16x8, xx), acc);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    __uint_as_float(val[j]), __uint_as_float(x.w[j]), acc, 0, 0, 0);
            return acc;
        }
    };

    if (ONE) copy(0);
    int first = 0, held = -1;  // part a turn starts with, and the one in LDS
    const int64_t tiles = (a.M + 15) / 16;
    for (int64_t tile0 = static_cast<int64_t>(blockIdx.x) * TR; tile0 < tiles;
         tile0 += static_cast<int64_t>(gridDim.x) * TR) {
        const uint32_t *rbits[TR];
        const uint32_t *rs0[TR];
        f32x4 acc[TR][BT];
#pragma unroll
        for (int r = 0; r < TR; ++r) {
            int64_t row = (tile0 + r) * 16 + l16;
            row = row < a.M ? row : a.M - 1;  // (not stored)
            rbits[r] = a.bits + row * a.runs * K;
            rs0[r] = a.s0 + row * a.bpr;
#pragma unroll
            for (int t = 0; t < BT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        if constexpr (ONE) {
            // x is asked for kAhead steps before its use, the words a unit before
            constexpr int kAhead = Sh::kAhead;
            uint32_t w[K + 1];
            Piece x[kAhead + 1][BT];
            const uint32_t s_end = u_end * 4 < a.runs ? u_end * 4 : a.runs;
            auto ask = [&](uint32_t s, Piece (&to)[BT]) {
                if (s < s_end) {
#pragma unroll
                    for (int t = 0; t < BT; ++t) to[t] = read_x(s, t);
                }
            };
            if (u_begin < u_end) {
                request(rbits[0], rs0[0], u_begin, w);
#pragma unroll
                for (int s = 0; s < kAhead; ++s) ask(u_begin * 4 + s, x[s]);
            }
            for (uint32_t u = u_begin; u < u_end; ++u) {
                uint32_t n[4][C::NW];
                align(w, n);
                // (the last turn asks for its own unit again)
                request(rbits[0], rs0[0], u + 1 < u_end ? u + 1 : u, w);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    ask(u * 4 + s + kAhead, x[(s + kAhead) % (kAhead + 1)]);
                    if (u * 4 + s < s_end) {
                        uint32_t val[kWords] = {};
                        decode(n[s], 0u, val);
#pragma unroll
                        for (int t = 0; t < BT; ++t)
                            acc[0][t] = multiply(val, x[s % (kAhead + 1)][t], acc[0][t]);
                    }
                }
            }
        } else {
            for (uint32_t k0 = 0; k0 < most; k0 += UN) {
                uint32_t n[TR][UN][4][C::NW];
                uint32_t val[TR][UN][4][kWords];
#pragma unroll
                for (int r = 0; r < TR; ++r)
#pragma unroll
                    for (int u = 0; u < UN; ++u) {
                        uint32_t w[K + 1];
                        request(rbits[r], rs0[r], u_begin + k0 + u, w);
                        align(w, n[r][u]);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int j = 0; j < kWords; ++j) val[r][u][s][j] = 0u;
                    }
                for (int v = 0; v < a.parts; ++v) {
                    const int p = first == 0 ? v : a.parts - 1 - v;
                    if (p != held) {
                        __syncthreads();  // the previous part is done with
                        copy(p);
                        held = p;
                    }
                    const uint32_t base = static_cast<uint32_t>(p) * dummy;
#pragma unroll
                    for (int r = 0; r < TR; ++r)
#pragma unroll
                        for (int u = 0; u < UN; ++u)
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                // (the states are extracted again for every part, one
                                // instruction each, rather than kept in registers)
#pragma unroll
                                for (int i = 0; i < C::NW; ++i)
                                    asm volatile("" : "+v"(n[r][u][s][i]));
                                decode(n[r][u][s], base, val[r][u][s]);
                                // (all chunks' reads at once do not fit the registers)
                                __builtin_amdgcn_sched_barrier(0);
                            }
                }
                first = first == 0 ? a.parts - 1 : 0;  // the next turn starts with this one
#pragma unroll
                for (int u = 0; u < UN; ++u)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t at = (u_begin + k0 + u) * 4 + s;
                        if (u_begin + k0 + u < u_end && at < a.runs) {
#pragma unroll
                            for (int t = 0; t < BT; ++t) {
                                const Piece x = read_x(at, t);
#pragma unroll
                                for (int r = 0; r < TR; ++r)
                                    acc[r][t] = multiply(val[r][u][s], x, acc[r][t]);
                            }
                        }
                    }
            }
        }
        // acc[r][t]: rows 4 g .. 4 g + 3 of the tile, row t 16 + l16 of x
#pragma unroll
        for (int q0 = 0; q0 < TR; q0 += kSumsR)
#pragma unroll
            for (int t0 = 0; t0 < BT; t0 += kSums) {
                __syncthreads();  // the previous sums are read
#pragma unroll
                for (int r = 0; r < kSumsR; ++r)
#pragma unroll
                    for (int t = 0; t < kSums; ++t)
                        *reinterpret_cast<f32x4 *>(
                            red + (((wave * kSumsR + r) * kSums + t) * 16 + l16) * 16 + g * 4) =
                            acc[q0 + r][t0 + t];
                __syncthreads();
                for (int o = tid; o < kSumsR * kSums * 256; o += kThreads) {
                    float sum = red[o];
#pragma unroll
                    for (int v = 1; v < kSmallWaves; ++v)
                        sum += red[v * kSumsR * kSums * 256 + o];
                    const int r = q0 + o / (kSums * 256), i = o % (kSums * 256);
                    epi.put_one(t0 * 16 + i / 16, (tile0 + r) * 16 + i % 16, sum);
                }
            }
    }
}

// ---------------------------------------------------------------- incoming gradient

struct SlopeArgs {
    const void *dy;
    int64_t B, M, lddy;
    const float *scale;      // row scale, or NULL
    const int8_t *zq;        // pre-activation checkpoint, or NULL (no activation)
    const uint8_t *ze;
    int64_t ldz;
    int64_t ld;              // of the result: a multiple of 8, columns past M are zeros
    float *part;             // [slabs][M] sums of dy act'(z) over a slab's rows, or NULL
    int64_t rows_per_slab;
    // fp16 in two terms: the largest |scale| is among tops[0 .. ntops - 1] (bit patterns; 1
    // without), and the power of two that out is to be multiplied by goes to *exponent
    const uint32_t *tops;
    int ntops;
    int *exponent;
};

// tops[block] = largest finite |scale[i]| of the block's share, as a bit pattern.
constexpr int kTops = 64;
__global__ __launch_bounds__(256) void scale_top_kernel(const float *__restrict__ scale,
                                                        int64_t M, uint32_t *__restrict__ tops) {
    __shared__ uint32_t red[4];
    uint32_t top = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < M;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const uint32_t m = __float_as_uint(scale[i]) & 0x7FFFFFFFu;
        if (m < 0x7F800000u && m > top) top = m;
    }
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(top, d);
        top = top > o ? top : o;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 4; ++w) top = top > red[w] ? top : red[w];
        tops[blockIdx.x] = top;
    }
}

// out = dy act'(z) scale in T, or in two terms of T; part = sums over a slab's rows of
// dy act'(z), in fp32 (each of the four waves adds every fourth row, then the four sums in
// order).  Eight columns per thread: memory-bound but for gelu.
//   Two terms hold a number x as high = T(x), low = T((x - high) 2^kLowShift): half(T)^2 of x.
// fp16 takes x = dy act'(z) scale 2^-e with |scale 2^-e| in [1/4, 1/2) for the largest |scale|,
// so |x| stays below 1.13 / 2 of fp16's largest number, and what low cannot hold is below 2^-36.
template <typename T, int ACT, int TERMS>
__global__ __launch_bounds__(256) void slope_kernel(SlopeArgs a, T *__restrict__ out,
                                                    T *__restrict__ out_low) {
    constexpr int kLow = gemm::kLowShift<T>;
    constexpr bool kTwo = TERMS == 2;
    constexpr float kBig = 1 << kLow;
    __shared__ float red[4][8][65];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int exponent = 0;
    if constexpr (TERMS == 2 && kLow != 0) {
        uint32_t top = a.tops ? (lane < a.ntops ? a.tops[lane] : 0u) : __float_as_uint(1.0f);
        for (int d = 32; d; d >>= 1) {
            const uint32_t o = __shfl_xor(top, d);
            top = top > o ? top : o;
        }
        // top below 2^(its exponent field - 126) (subnormals: the smallest normal exponent's)
        const int field = static_cast<int>(top >> 23);
        exponent = (field > 1 ? field : 1) - 125;
        if (a.exponent && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            *a.exponent = exponent;
    }
    const int64_t c0 = (static_cast<int64_t>(blockIdx.x) * 64 + lane) * 8;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.rows_per_slab;
    const int64_t r1 = r0 + a.rows_per_slab < a.B ? r0 + a.rows_per_slab : a.B;
    const T *dy = static_cast<const T *>(a.dy);
    const int64_t groups = (a.M + 31) / 32;
    const int left = a.M - c0 < 8 ? static_cast<int>(a.M - c0) : 8;  // may be <= 0
    float sum[8], sc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sum[e] = 0.0f;
        // (0 past M: a power of two times 1 may be an infinity)
        sc[e] = e < left ? (a.scale ? a.scale[c0 + e] : 1.0f) : 0.0f;
        if constexpr (TERMS == 2 && kLow != 0)
            sc[e] = __builtin_amdgcn_ldexpf(sc[e], kLow - exponent);
    }
    if (c0 < a.ld) {
#pragma unroll 2
        for (int64_t r = r0 + w; r < r1; r += 4) {
            Packed<T> d;
            Packed<int8_t> z;
            int ez = 0;
            if (left == 8) {
                d = *reinterpret_cast<const Packed<T> *>(dy + r * a.lddy + c0);
                if constexpr (ACT != TCQ_ACT_NONE)
                    z = *reinterpret_cast<const Packed<int8_t> *>(a.zq + r * a.ldz + c0);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d.v[e] = e < left ? dy[r * a.lddy + c0 + e] : static_cast<T>(0.0f);
                    if constexpr (ACT != TCQ_ACT_NONE)
                        z.v[e] = e < left ? a.zq[r * a.ldz + c0 + e] : static_cast<int8_t>(0);
                }
            }
            if constexpr (ACT != TCQ_ACT_NONE) ez = left > 0 ? a.ze[r * groups + c0 / 32] : 0;
            struct alignas(8 * sizeof(T)) Eight { T v[8]; } o, low;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float g = static_cast<float>(d.v[e]);
                if constexpr (ACT != TCQ_ACT_NONE)
                    if (e < left) g = act_grad<ACT, sizeof(T) == 4>(g, code_value(z.v[e], ez));
                sum[e] += g;
                const float x = g * sc[e];  // (two terms: times 2^kLow)
                // Every step from x on is exact but for the two roundings to T.  (The compiler
                // takes the product before a rounding to fp16 exactly where it can, in one
                // use of x and not in another: with x - T(x) the low term belonged to
                // another high one where x is halfway.)
                o.v[e] = static_cast<T>(kTwo ? x * (1.0f / kBig) : x);
                if constexpr (TERMS == 2) {
                    const float high = static_cast<float>(o.v[e]);
                    const float rest = __builtin_fmaf(high, -kBig, x);
                    // an infinity or a NaN is the high term's alone
                    low.v[e] = static_cast<T>(__builtin_fabsf(high) < __builtin_inff() ? rest : 0.0f);
                }
            }
            if (out) {
                *reinterpret_cast<Eight *>(out + r * a.ld + c0) = o;
                if constexpr (TERMS == 2) *reinterpret_cast<Eight *>(out_low + r * a.ld + c0) = low;
            }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) red[w][e][lane] = sum[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 512; i += 256) {
        const int l = i >> 3, e = i & 7;
        const int64_t c = static_cast<int64_t>(blockIdx.x) * 512 + i;
        if (c < a.M)
            a.part[static_cast<int64_t>(blockIdx.y) * a.M + c] =
                ((red[0][e][l] + red[1][e][l]) + red[2][e][l]) + red[3][e][l];
    }
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

__global__ __launch_bounds__(256) void slab_sum_kernel(const float *__restrict__ part,
                                                       int64_t slabs, int64_t M,
                                                       float *__restrict__ sum) {
    slab_sum(part, slabs, M, sum, blockIdx.x);
}

// slab_sum and act_unpack, which know nothing of each other, side by side in one launch (509 x
// 2048 and 4096 x 4096 in 16 bits: 4.1 and 14.5 us, as two 5.9 and 18.9): the first `sums`
// workgroups take the sums.
template <typename T, bool SMALL>
__global__ __launch_bounds__(256) void slab_sum_unpack_kernel(const float *__restrict__ part,
                                                              int64_t slabs, int64_t M,
                                                              float *__restrict__ sum,
                                                              uint32_t sums, UnpackArgs a,
                                                              T *__restrict__ out) {
    if (blockIdx.x < sums)
        slab_sum(part, slabs, M, sum, blockIdx.x);
    else
        act_unpack<T, SMALL>(a, out, blockIdx.x - sums, gridDim.x - sums);
}

// ---------------------------------------------------------------- host side

template <typename T>
bool four_aligned(const T *p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T))) == 0 && ld % 4 == 0;
}

// Whether rows of p can be read 16 bytes at a time by the product: aligned, and the
// contiguous extent a whole number of 16-byte pieces.
bool sixteen_aligned(const void *p, int64_t ld, int64_t extent, size_t size) {
    const int64_t per = static_cast<int64_t>(16 / size);
    // (a tile's byte offsets fit 32 bits: 256 rows of at most 2^21 values)
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % per == 0 && extent % per == 0 &&
           ld <= TCQ_LINEAR_MAX_DIM;
}

unsigned grid_for(int64_t work, int64_t per, int64_t most) {
    int64_t g = (work + per - 1) / per;
    if (g > most) g = most;
    return static_cast<unsigned>(g < 1 ? 1 : g);
}

// Row slabs of the incoming gradient's pass: about 1024 workgroups of 512 columns, at least
// eight rows each.
int64_t slope_slabs(int64_t B, int64_t M) {
    const int64_t cols = (M + 511) / 512;
    int64_t s = cols > 0 ? (1024 + cols - 1) / cols : 1;
    if (s > (B + 7) / 8) s = (B + 7) / 8;
    return s < 1 ? 1 : s;
}

template <typename T, int TERMS>
const void *slope_kernel_of(int act) {
    // (silu and gelu take two terms of a 16-bit type)
    if constexpr (sizeof(T) == 4 || TERMS == 2) {
        if (act == TCQ_ACT_SILU)
            return reinterpret_cast<const void *>(slope_kernel<T, TCQ_ACT_SILU, TERMS>);
        if (act == TCQ_ACT_GELU)
            return reinterpret_cast<const void *>(slope_kernel<T, TCQ_ACT_GELU, TERMS>);
    }
    if (act == TCQ_ACT_RELU)
        return reinterpret_cast<const void *>(slope_kernel<T, TCQ_ACT_RELU, TERMS>);
    return reinterpret_cast<const void *>(slope_kernel<T, TCQ_ACT_NONE, TERMS>);
}

// Terms of a 16-bit type that the scaled gradient is held in: one where it is dy itself or zero.
int grad_terms(const LinearGrad &c) {
    return c.row_scale || c.act == TCQ_ACT_SILU || c.act == TCQ_ACT_GELU ? 2 : 1;
}

// Compute units of the current device, for grids whose workgroups share work in any number
// (asked on every call: devices of one process, such as partitions of one GPU, need not have
// the same count; gemm_plan's tiles and splits decide how sums are rounded, and do not ask).
int cu_count() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
        n > 0)
        return n;
    return 256;
}

// The chunk kernel of (kV, V), or nullptr.
template <typename T>
const void *chunk_kernel(int kv, int V, bool one) {
// (a 16-bit table of V = 1 always fits one part)
#define TCQ_CHUNK_CASE(KV_, V_)                                                           \
    if (kv == KV_ && V == V_) {                                                           \
        if constexpr (V_ > 1 || sizeof(T) == 4)                                           \
            if (!one)                                                                     \
                return reinterpret_cast<const void *>(decode_chunks_kernel<T, KV_, V_, false>); \
        return reinterpret_cast<const void *>(decode_chunks_kernel<T, KV_, V_, true>);    \
    }
    TCQ_CHUNK_CASE(1, 1)
    TCQ_CHUNK_CASE(2, 1)
    TCQ_CHUNK_CASE(2, 2)
    TCQ_CHUNK_CASE(3, 1)
    TCQ_CHUNK_CASE(4, 1)
    TCQ_CHUNK_CASE(4, 2)
    TCQ_CHUNK_CASE(4, 4)
    TCQ_CHUNK_CASE(6, 1)
    TCQ_CHUNK_CASE(6, 2)
    TCQ_CHUNK_CASE(8, 1)
    TCQ_CHUNK_CASE(8, 2)
    TCQ_CHUNK_CASE(8, 4)
#undef TCQ_CHUNK_CASE
    return nullptr;
}

// Raises the dynamic LDS limit of a kernel to all of a compute unit's.  Set on every launch: the
// attribute belongs to the function on the current device, and nothing is kept between
// calls.  Always the same number: with a call's own size, another thread's call of the same
// kernel with a smaller table could lower it before this one is launched.
hipError_t allow_lds(const void *kern) {
    return hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
}

template <typename T>
hipError_t decode_matrix(const CodedMatrix &w, T *out, int64_t ld, hipStream_t s) {
    if (w.M <= 0 || w.N <= 0) return hipSuccess;
    const int kv = w.k * w.V;
    const int nwords = (w.k * w.T + 31) / 32;
    const int64_t chunks = w.M * (w.N / 8);
    const size_t row = w.V * sizeof(T);
    const size_t table = row << w.L;
    const bool one = table <= kPartBytes;
    const void *kern = w.T % 8 == 0 && chunks < (int64_t{1} << 31) && table % 16 == 0
                           ? chunk_kernel<T>(kv, w.V, one)
                           : nullptr;
    if (kern) {
        ChunkArgs a{};
        a.bits = w.bits;
        a.s0 = w.s0;
        a.table = static_cast<const char *>(w.table);
        a.chunks = static_cast<uint32_t>(chunks);
        a.cpb = static_cast<uint32_t>(w.T / 8);
        a.cpb_log2 = -1;
        for (int b = 0; b < 16; ++b)
            if (a.cpb == (1u << b)) a.cpb_log2 = b;
        a.L = w.L;
        a.nwords = nwords;
        a.part_log2 = w.L;
        while ((row << a.part_log2) > kPartBytes) --a.part_log2;
        a.parts = 1 << (w.L - a.part_log2);
        a.vec = (reinterpret_cast<uintptr_t>(w.table) & 15) == 0;
        // the part, the row of zeros, and the room a partly filled wave of the copy writes
        const size_t lds = (row << a.part_log2) + 1024;
        const int64_t slots = static_cast<int64_t>(cu_count()) * (lds <= (72 << 10) ? 2 : 1);
        int64_t grid = (chunks + kChunkThreads - 1) / kChunkThreads;
        if (grid > slots) grid = slots;
        a.chunks_per_wg = static_cast<uint32_t>((chunks + grid - 1) / grid);
        grid = (chunks + a.chunks_per_wg - 1) / a.chunks_per_wg;
        // the fewest turns, the chunks spread evenly over them
        const int rt = one ? chunk_rows<T, true>() : chunk_rows<T, false>();
        const int64_t per = (a.chunks_per_wg + kChunkThreads - 1) / kChunkThreads;
        const int64_t turns = (per + rt - 1) / rt;
        a.rows = static_cast<int>((per + turns - 1) / turns);
        hipError_t e = allow_lds(kern);
        if (e != hipSuccess) return e;
        T *o = out;
        void *args[] = {&a, &o};
        e = hipLaunchKernel(kern, dim3(static_cast<unsigned>(grid)), dim3(kChunkThreads), args,
                            lds, s);
        return e != hipSuccess ? e : hipGetLastError();
    }
    const DecodeArgs a{w.bits, w.s0, w.table, w.M, w.N, ld, w.L, kv, w.V, w.T, nwords};
    hipLaunchKernelGGL(decode_matrix_kernel<T>, dim3(grid_for(w.M * (ld / 8), 256, 1 << 20)),
                       dim3(256), 0, s, a, out);
    return hipGetLastError();
}

template <typename T>
LayerEpilogue<T> layer_epilogue(const CodedMatrix &w, const LinearCall &c) {
    LayerEpilogue<T> epi{};
    epi.scale = c.row_scale;
    epi.bias = c.bias;
    epi.res = static_cast<const T *>(c.residual);
    epi.y = static_cast<T *>(c.y);
    epi.pre = static_cast<T *>(c.pre);
    epi.ldr = c.ldr;
    epi.ldy = c.ldy;
    epi.ldp = c.ldp;
    epi.I = c.B;
    epi.J = w.M;
    epi.act = c.act;
    epi.vec_y = four_aligned(epi.y, c.ldy);
    epi.vec_r = four_aligned(epi.res, c.ldr);
    epi.vec_p = four_aligned(epi.pre, c.ldp);
    return epi;
}

template <typename T, int BT, bool ONE>
const void *small_kernel_of(int kv, int V) {
// (a 16-bit table of V = 1 always fits one part, and one of several goes up to 64 rows)
#define TCQ_SMALL_CASE(KV_, V_)                                      \
    if constexpr (ONE || sizeof(T) == 4 || (V_ > 1 && BT <= 4))      \
        if (kv == KV_ && V == V_)                      \
            return reinterpret_cast<const void *>(small_kernel<T, KV_, V_, BT, ONE>);
    TCQ_SMALL_CASE(1, 1)
    TCQ_SMALL_CASE(2, 1)
    TCQ_SMALL_CASE(2, 2)
    TCQ_SMALL_CASE(3, 1)
    TCQ_SMALL_CASE(4, 1)
    TCQ_SMALL_CASE(4, 2)
    TCQ_SMALL_CASE(4, 4)
#undef TCQ_SMALL_CASE
    return nullptr;
}

template <typename T, int BT>
hipError_t forward_small(const CodedMatrix &w, const LinearCall &c, char *ws, hipStream_t s) {
    SmallArgs a{};
    a.bits = w.bits;
    a.s0 = w.s0;
    a.table = static_cast<const char *>(w.table);
    a.x = c.x;
    a.B = c.B;
    a.ldx = c.ldx;
    a.M = w.M;
    a.runs = static_cast<uint32_t>(w.N / 32);
    a.bpr = static_cast<uint32_t>(w.N / w.T);
    a.rpb = static_cast<uint32_t>(w.T / 32);
    a.rpb_log2 = -1;
    for (int b = 0; b < 16; ++b)
        if (a.rpb == (1u << b)) a.rpb_log2 = b;
    a.L = w.L;
    const size_t row = w.V * sizeof(T);
    int plog = w.L;
    while ((row << plog) > kPartBytes) --plog;
    a.part_bytes = static_cast<int>(row << plog);
    a.parts = 1 << (w.L - plog);
    a.vec = (reinterpret_cast<uintptr_t>(w.table) & 15) == 0;
    hipError_t e;
    if constexpr (BT > 1) {
        const int64_t pieces =
            static_cast<int64_t>(a.runs) * BT * static_cast<int64_t>(sizeof(T) / 2) * 64;
        hipLaunchKernelGGL((pack_rows_kernel<T, BT>), dim3(grid_for(pieces, 256, 1 << 16)),
                           dim3(256), 0, s, static_cast<const T *>(c.x), c.B, c.ldx, pieces,
                           reinterpret_cast<uint4 *>(ws));
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.x = ws;
    }
    const int kv = w.k * w.V;
    const bool one = a.parts == 1;
    const int tr = one ? SmallShape<T, BT, true>::TR : SmallShape<T, BT, false>::TR;
    const size_t sums = static_cast<size_t>(kSmallWaves) * 1024 *
                        (one ? SmallShape<T, BT, true>::kSums : SmallShape<T, BT, false>::kSums);
    // The sums lie behind the table: behind the 1 KiB that a partly filled wave of the copy
    // of a small one writes, or the row of zeros after a part.
    a.red = one ? (a.part_bytes < 1024 ? 1024 : a.part_bytes) : a.part_bytes + 64;
    const size_t lds = a.red + sums;
    const void *kern = one ? small_kernel_of<T, BT, true>(kv, w.V)
                           : small_kernel_of<T, BT, false>(kv, w.V);
    e = allow_lds(kern);
    if (e != hipSuccess) return e;
    const int64_t turns = ((w.M + 15) / 16 + tr - 1) / tr;
    const int64_t slots = static_cast<int64_t>(cu_count()) * (lds <= (80 << 10) ? 2 : 1);
    LayerEpilogue<T> epi = layer_epilogue<T>(w, c);
    void *args[] = {&a, &epi};
    e = hipLaunchKernel(kern,
                        dim3(static_cast<unsigned>(turns < slots ? turns : slots)),
                        dim3(kSmallWaves * 64), args, lds, s);
    return e != hipSuccess ? e : hipGetLastError();
}

template <typename T>
hipError_t forward(const CodedMatrix &w, const LinearCall &c, char *ws, hipStream_t s) {
    const LinearLayout lay = linear_layout(sizeof(T), c.B, w.M, w.N);
    switch (linear_small(sizeof(T), c.B, w.N, w.L, w.k, w.V, w.T)) {
        case 1: return forward_small<T, 1>(w, c, ws, s);
        case 2: return forward_small<T, 2>(w, c, ws, s);
        case 4: return forward_small<T, 4>(w, c, ws, s);
        case 8: return forward_small<T, 8>(w, c, ws, s);
        default: break;
    }
    T *W = reinterpret_cast<T *>(ws + lay.matrix);
    hipError_t e = decode_matrix(w, W, lay.ldn, s);
    if (e != hipSuccess) return e;
    const T *x = static_cast<const T *>(c.x);
    int64_t ldx = c.ldx, K = w.N;
    if (w.N > 0 && !sixteen_aligned(x, ldx, w.N, sizeof(T))) {
        T *st = reinterpret_cast<T *>(ws + lay.rows);
        hipLaunchKernelGGL(stage_kernel<T>, dim3(grid_for(c.B * lay.ldn, 1024, 1 << 16)),
                           dim3(256), 0, s, x, c.B, w.N, ldx, st, lay.ldn);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        x = st;
        ldx = lay.ldn;
        K = lay.ldn;
    }
    const LayerEpilogue<T> epi = layer_epilogue<T>(w, c);
    const Operand<T> A{x, ldx, c.B, K};
    const Operand<T> Bm{W, lay.ldn, w.M, K};
    return launch_gemm<T, false, false, 1>(A, Bm, lay.forward, epi, ws + lay.sums, s);
}

template <typename T, int TERMS>
hipError_t backward(const CodedMatrix &w, const LinearGrad &c, char *ws, hipStream_t s) {
    const LinearLayout lay =
        linear_grad_layout(sizeof(T), c.B, w.M, w.N, c.dx, c.dw, c.dbias, TERMS);
    hipError_t e;
    T *S = reinterpret_cast<T *>(ws + lay.grad);
    T *low = reinterpret_cast<T *>(ws + lay.low);
    // the power of two that fp16 sums are to be multiplied by
    uint32_t *tops = reinterpret_cast<uint32_t *>(ws + lay.tops);
    int *exponent =
        TERMS == 2 && gemm::kLowShift<T> != 0 ? reinterpret_cast<int *>(tops + kTops) : nullptr;
    const int64_t slabs = slope_slabs(c.B, w.M);
    if (c.B > 0 && w.M > 0) {
        SlopeArgs a{};
        a.dy = c.dy;
        a.B = c.B;
        a.M = w.M;
        a.lddy = c.lddy;
        a.scale = c.row_scale;
        a.zq = c.zq;
        a.ze = c.ze;
        a.ldz = c.ldz;
        a.ld = lay.ldm;
        a.part = c.dbias ? reinterpret_cast<float *>(ws + lay.part) : nullptr;
        a.rows_per_slab = (c.B + slabs - 1) / slabs;
        T *out = c.dx || c.dw ? S : nullptr;
        a.exponent = out ? exponent : nullptr;
        if (a.exponent && c.row_scale) {
            a.tops = tops;
            a.ntops = static_cast<int>(grid_for(w.M, 2048, kTops));
            hipLaunchKernelGGL(scale_top_kernel, dim3(static_cast<unsigned>(a.ntops)), dim3(256),
                               0, s, c.row_scale, w.M, tops);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        void *args[] = {&a, &out, &low};
        e = hipLaunchKernel(slope_kernel_of<T, TERMS>(c.act),
                            dim3(static_cast<unsigned>((lay.ldm / 8 + 63) / 64),
                                 static_cast<unsigned>(slabs)),
                            dim3(256), args, 0, s);
        if (e != hipSuccess) return e;
    }
    // x's checkpoint is unpacked for dw; the bias' sums go along in the same launch
    const bool unpack = c.dw && c.B > 0 && w.M > 0 && w.N > 0;
    const bool sum = c.dbias && w.M > 0;
    const float *part = reinterpret_cast<const float *>(ws + lay.part);
    T *X = reinterpret_cast<T *>(ws + lay.rows);
    const uint32_t sums = static_cast<uint32_t>((w.M + 63) / 64);
    if (unpack && sum) {
        const UnpackArgs a =
            unpack_args<T>(c.xq, c.ldxq, c.xe, c.B, w.N, lay.ldn, lay.ldn);
        const auto kern = a.ix.total < (int64_t{1} << 32) ? slab_sum_unpack_kernel<T, true>
                                                          : slab_sum_unpack_kernel<T, false>;
        hipLaunchKernelGGL(kern, dim3(sums + grid_for(a.ix.total, 256, 1 << 20)), dim3(256), 0,
                           s, part, slabs, w.M, c.dbias, sums, a, X);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else if (sum) {
        hipLaunchKernelGGL(slab_sum_kernel, dim3(sums), dim3(256), 0, s, part,
                           c.B > 0 ? slabs : 0, w.M, c.dbias);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else if (unpack) {
        e = launch_act_unpack(c.xq, c.ldxq, c.xe, c.B, w.N, dtype_of<T>(), X, lay.ldn, lay.ldn,
                              s);
        if (e != hipSuccess) return e;
    }
    const int64_t to_low = static_cast<int64_t>(lay.low) - static_cast<int64_t>(lay.grad);
    if (c.dx && c.B > 0 && w.N > 0) {
        T *W = reinterpret_cast<T *>(ws + lay.matrix);
        e = decode_matrix(w, W, lay.ldn, s);
        if (e != hipSuccess) return e;
        const PlainEpilogue<T> epi{static_cast<T *>(c.dx), c.lddx, c.B, w.N,
                                   four_aligned(static_cast<T *>(c.dx), c.lddx),
                                   c.B > 0 && w.M > 0 ? exponent : nullptr};
        const Operand<T> A{S, lay.ldm, c.B, w.M > 0 ? lay.ldm : 0, to_low};
        // (columns past N are zeros and not stored; rows past M read as zeros)
        const Operand<T> Bm{W, lay.ldn, lay.ldn, w.M};
        e = launch_gemm<T, false, true, TERMS>(A, Bm, lay.dx, epi, ws + lay.sums, s);
        if (e != hipSuccess) return e;
    }
    if (c.dw && w.M > 0 && w.N > 0) {
        const PlainEpilogue<T> epi{static_cast<T *>(c.dw), c.lddw, w.M, w.N,
                                   four_aligned(static_cast<T *>(c.dw), c.lddw),
                                   c.B > 0 ? exponent : nullptr};
        const Operand<T> A{S, lay.ldm, lay.ldm, c.B, to_low};
        const Operand<T> Bm{X, lay.ldn, lay.ldn, c.B};
        e = launch_gemm<T, true, true, TERMS>(A, Bm, lay.dw, epi, ws + lay.sums, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
hipError_t backward(const CodedMatrix &w, const LinearGrad &c, char *ws, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (grad_terms(c) == 2) return backward<T, 2>(w, c, ws, s);
    }
    return backward<T, 1>(w, c, ws, s);
}

size_t pad8(int64_t n) { return static_cast<size_t>((n + 7) / 8 * 8); }

}  // namespace

// Up to 128 rows are decoded inside the product, 64 where a 16-bit table has several parts
// (us per call, inside at the limit / through the workspace with one row more).  4096 x 4096 in
// bf16: 22 / 32; 14336 x 4096 V=2 in bf16: 52 / 69; 4096 x 4096 in fp32: 67 / 80.  Beyond it,
// inside / through the workspace: 256 rows of the first 40 / 35, 128 rows of the second 78 / 72.
int linear_small(size_t size, int64_t B, int64_t N, int L, int k, int V, int T) {
    const int kv = k * V;
    if (N <= 0 || T % 32 != 0 || kv > 4 || (V != 1 && V != 2 && V != 4)) return 0;
    const size_t table = (V * size) << L;
    if (table % 16 != 0) return 0;  // the table's copy moves 16 bytes at a time
    const bool one = table <= kPartBytes;
    if (B > (size == 4 || one ? 128 : 64)) return 0;
    return B <= 16 ? 1 : (B <= 32 ? 2 : (B <= 64 ? 4 : 8));
}

size_t linear_small_bytes(size_t size, int64_t N, int bt) {
    return bt > 1 ? static_cast<size_t>(16 * bt) * N * size : 0;
}

// Tile and splits of an I x J product over K.  The choice depends on sizes alone (and on
// the 256 compute units of the part this library is built for), so the workspace query
// and the call agree.
//   64 x 128 tiles with two stages run three to a compute unit.  Where there are few, k is
// split into about 512 workgroups and the shares, in fp32, are added by a second kernel (512 x
// 4096 x 4096 in bf16: 57 us per call unsplit, 45 split; 160 rows: 40 and 32).  A split has at
// least 4 steps (with at least 2 / 4 / 8, bf16, in a graph: 300 x 1024 x 1024 18.0 / 15.3 / 15.8
// us, 150 x 2048 x 512 14.4 / 13.8 / 14.8), and there are at most 16 (with 8 / 16 / 32: 200 x 256 x
// 14336 34.3 / 29.2 / 30.9 us in bf16, 84 / 56 / 46 in fp32).
//   16-bit types also have 256 x 256 tiles (the ring) and 128 x 128 ones (four stages), one
// to a compute unit.  Tiles come in rounds of 256; what a round costs, once and per step of
// k, was fitted to calls with all three forced on the same shapes, and the cheapest is taken
// (566 x 6912 x 2176 in bf16: 56 us per call with 64 x 128, 76 with 128 x 128, 70 with
// 256 x 256; 2176 x 6912 x 576: 57, 72 and 40; 1024 x 4096 x 4096: 67, 63 and 99).
//   fp32 has 128 x 128 ones with two stages, two to a compute unit, which split a fragment's
// values for twice as many products but leave more of the card idle in a last round (566 x
// 6912 x 2176: 152 us per call with 64 x 128, 200 with 128 x 128; 2176 x 6912 x 576: 145 and
// 127).
//   128 x 128 tiles are split over k too, into 256 workgroups of a 16-bit type and 512 in fp32,
// where two share a compute unit (1000 x 2048 x 2048 as 64 x 128 and 128 x 128, both split: 39
// and 34 us per call in bf16, 82 and 75 in fp32, where 256 workgroups take 86; 200 x 14336 x
// 4096 in fp32: 330 and 268; 333 x 2048 x 2048: 30 and 32 in bf16, 51 and 51 in fp32).
constexpr int64_t kCus = 256, kMostSplits = 16, kLeastSteps = 4;

int64_t gemm_steps(size_t size, int64_t K, int terms) {
    const int64_t step = gemm::kStepBytes / static_cast<int64_t>(size);
    return (K + step - 1) / step * terms;
}

GemmPlan gemm_plan(size_t size, int64_t I, int64_t J, int64_t K, int terms) {
    const auto tiles = [&](int64_t ti, int64_t tj) {
        return ((I + ti - 1) / ti) * ((J + tj - 1) / tj);
    };
    const auto rounds = [&](int64_t n) { return static_cast<double>((n + kCus - 1) / kCus); };
    GemmPlan p{};
    p.steps = static_cast<int>(gemm_steps(size, K, terms));
    p.part_ld = (J + 3) / 4 * 4;
    // n tiles with k split into about `most` workgroups
    const auto split = [&](int tile, int64_t n, int64_t most) {
        GemmPlan q = p;
        q.tile = tile;
        int64_t s = n > 0 ? most / n : 1;
        if (s > q.steps / kLeastSteps) s = q.steps / kLeastSteps;
        if (s > kMostSplits) s = kMostSplits;
        if (s < 1) s = 1;
        q.steps_per_split = static_cast<int>((q.steps + s - 1) / s);
        q.splits = q.steps_per_split > 0
                       ? (q.steps + q.steps_per_split - 1) / q.steps_per_split
                       : 1;
        q.part_bytes = q.splits > 1 ? static_cast<size_t>(q.splits) * I * q.part_ld * 4 : 0;
        return q;
    };
    // us; the shares are read at about 4 TB/s, and their kernel takes 3 more
    const auto join = [](const GemmPlan &q) {
        return q.splits > 1 ? 3.0 + q.part_bytes / 4e6 : 0.0;
    };
    GemmPlan best{};
    double least = 0.0;
    const auto take = [&](const GemmPlan &q, double us) {
        us += join(q);
        if (best.splits != 0 && us >= least) return;
        least = us;
        best = q;
    };
    const int64_t n64 = tiles(64, 128), n128 = tiles(128, 128);
    const GemmPlan s64 = split(kTile64, n64, 2 * kCus);
    const double r = rounds(n64 * s64.splits);
    if (size == 2) {
        take(s64, 4.0 + 1.5 * r + 0.33 * (r < 3 ? 3 : r) * s64.steps_per_split);
        take(split(kTile128, n128, n128), 4.0 + rounds(n128) * (5.0 + 0.8 * p.steps));
        take(split(kTile256, 1, 1), 7.0 + rounds(tiles(256, 256)) * (12.0 + 1.4 * p.steps));
        const GemmPlan q = split(kTile128, n128, kCus);
        if (q.splits > 1) take(q, 9.0 + 0.8 * q.steps_per_split);
    } else {
        take(s64, 4.0 + r * (1.5 + 0.88 * s64.steps_per_split));
        // rounds of two to a compute unit, the last of one where that is enough
        const auto pairs = [&](const GemmPlan &q) {
            const int64_t n = n128 * q.splits, left = n % (2 * kCus);
            return 4.0 + (n / (2 * kCus) + (left > kCus)) * (8.0 + 2.6 * q.steps_per_split) +
                   (left > 0 && left <= kCus ? 4.0 + 2.0 * q.steps_per_split : 0.0);
        };
        const GemmPlan whole = split(kTile128, n128, n128), q = split(kTile128, n128, 2 * kCus);
        take(whole, pairs(whole));
        if (q.splits > 1) take(q, pairs(q));
    }
    return best;
}

// Room for a product's shares: at least the plan's part_bytes, and never less for a larger I or
// K, although a larger product may not be split at all, so that a workspace of one batch
// serves every smaller one.  n tiles of 64 x 128 or 128 x 128 are split into at most 2 kCus or
// kCus workgroups (2 kCus in fp32), so no plan's shares are larger than theirs.
size_t gemm_shares(size_t size, int64_t I, int64_t J, int64_t K, int terms) {
    const int64_t most = size == 2 ? kCus * 128 * 128 : 2 * kCus * 128 * 128;
    static_assert(2 * kCus * 64 * 128 <= kCus * 128 * 128, "the larger of the two");
    int64_t s = gemm_steps(size, K, terms) / kLeastSteps;
    if (s > kMostSplits) s = kMostSplits;
    if (s < 2) return 0;
    const int64_t values = s * I * ((J + 3) / 4 * 4);
    return static_cast<size_t>(values < most ? values : most) * sizeof(float);
}

LinearLayout linear_layout(size_t size, int64_t B, int64_t M, int64_t N) {
    LinearLayout l{};
    l.ldn = static_cast<int64_t>(pad8(N));
    l.matrix = 0;
    l.rows = align_up(static_cast<size_t>(M) * l.ldn * size, 256);
    l.sums = l.rows + align_up(static_cast<size_t>(B) * l.ldn * size, 256);
    l.forward = gemm_plan(size, B, M, l.ldn, 1);
    l.bytes = l.sums + align_up(gemm_shares(size, B, M, l.ldn, 1), 256);
    return l;
}

LinearLayout linear_grad_layout(size_t size, int64_t B, int64_t M, int64_t N, bool dx, bool dw,
                                bool dbias, int terms) {
    LinearLayout l{};
    l.ldn = static_cast<int64_t>(pad8(N));
    l.ldm = static_cast<int64_t>(pad8(M));
    size_t off = 0;
    l.matrix = off;
    if (dx) off += align_up(static_cast<size_t>(M) * l.ldn * size, 256);
    l.grad = off;
    if (dx || dw) off += align_up(static_cast<size_t>(B) * l.ldm * size, 256);
    // (the query does not know whether a call needs the second term)
    l.low = off;
    if ((dx || dw) && size == 2) off += align_up(static_cast<size_t>(B) * l.ldm * size, 256);
    l.tops = off;
    if ((dx || dw) && size == 2) off += align_up((kTops + 1) * sizeof(uint32_t), 256);
    l.rows = off;
    if (dw) off += align_up(static_cast<size_t>(B) * l.ldn * size, 256);
    l.part = off;
    if (dbias) off += align_up(static_cast<size_t>(slope_slabs(B, M)) * M * sizeof(float), 256);
    l.sums = off;  // (the two products run one after the other)
    l.dx = gemm_plan(size, B, l.ldn, M, terms);
    l.dw = gemm_plan(size, l.ldm, l.ldn, B, terms);
    const int most = size == 2 ? 2 : 1;
    const size_t gx = dx ? gemm_shares(size, B, l.ldn, M, most) : 0;
    const size_t gw = dw ? gemm_shares(size, l.ldm, l.ldn, B, most) : 0;
    off += align_up(gx > gw ? gx : gw, 256);
    l.bytes = off;
    return l;
}

hipError_t launch_linear(const CodedMatrix &w, const LinearCall &c, char *ws, hipStream_t s) {
    switch (c.dtype) {
        case TCQ_F32: return forward<float>(w, c, ws, s);
        case TCQ_F16: return forward<_Float16>(w, c, ws, s);
        default: return forward<__bf16>(w, c, ws, s);
    }
}

hipError_t launch_linear_grad(const CodedMatrix &w, const LinearGrad &c, char *ws,
                              hipStream_t s) {
    switch (c.dtype) {
        case TCQ_F32: return backward<float>(w, c, ws, s);
        case TCQ_F16: return backward<_Float16>(w, c, ws, s);
        default: return backward<__bf16>(w, c, ws, s);
    }
}

}  // namespace tcq
