// Tiled matrix product of the coded linear layer on the matrix cores (device code).
//
//   D[i][j] = sum_k A(i, k) B(j, k),      i < I, j < J
//
// for operands of one type (float, _Float16 or __bf16) whose products are summed in fp32.
// Each operand is stored either with k contiguous (X[row][k], "row-major in k") or with its
// rows contiguous (X[k][row], "k-major"); the forward product, the input's gradient and
// the matrix's gradient are the three combinations, so no operand is transposed in memory.
//
// A workgroup computes a TI x TJ tile of D over steps of 128 bytes of k per row (64 16-bit or
// 32 fp32 values).  Both operand tiles of a step go from global memory straight into LDS
// (buffer_load_dwordx4 ... lds), in NB stages: the loads of the next NB - 1 steps are in
// flight while a step is multiplied (or in a ring of five pieces).  The stages are separate
// LDS variables, and the loop is unrolled over them, so that the compiler sees that reads of
// one cannot touch the loads into the others and does not wait for those.  Rows past I or J
// and k past K read as zeros: a buffer descriptor ends with the operand's last row, and lanes
// past K get an offset past its end.
//
// LDS layout.  A k-contiguous tile has rows of 128 bytes, eight 16-byte chunks; chunk c of
// row r sits in slot c ^ ((r >> 1) & 7), so the 16 rows that a fragment read touches lie in
// 16 different 16-byte columns of the 256 bytes the banks span.  A k-major tile has one row
// of T values per k; for 16-bit types its 32-byte units (16 columns, what one transposing
// read takes from a row) are permuted by the key (k & 3) | (k >> 3 & 1) << 2, which sends
// the eight k rows that two groups of 16 lanes read together to eight different units.
// The permutation is applied to the global address of each lane, since LDS-direct loads
// write LDS linearly.
//
// The matrix instruction takes B(j, .) as its first operand, so a lane ends up with four
// consecutive j of one row i: outputs leave in 8- or 16-byte pieces.
//
// A 16-bit operand A can be held in two terms, A = high + 2^-kLowShift low, each stored like A
// (TERMS = 2).  The steps then run over k twice, first with the low term, and between the two
// the sums are scaled by 2^-kLowShift, which is exact: no second set of sums is needed.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace tcq {
namespace gemm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// One operand in global memory.  rows: valid rows (I or J); k: valid k.  For k-contiguous
// storage element (row, kk) is at p[row * ld + kk], for k-major storage at p[kk * ld + row].
// p is 16-byte aligned, ld * sizeof(T) a multiple of 16, and the contiguous extent (k, or
// rows) a multiple of 16 bytes too.
template <typename T>
struct Operand {
    const T *p;
    int64_t ld;
    int64_t rows;
    int64_t k;
    int64_t low = 0;  // bytes from p to the low term, where there are two
};

// An fp16 remainder may fall below the type's smallest number, so it is held 2^11 times as
// large (at most 16 of a number below 65504, 2^15 then); bf16 has the exponents of fp32.
template <typename T>
constexpr int kLowShift = __is_same(T, _Float16) ? 11 : 0;

constexpr int kStepBytes = 128;  // bytes of k per row and step
constexpr int kPastEnd = -1;     // a step that reads as zeros

template <typename T>
struct Traits;
template <>
struct Traits<float> {
    static constexpr int kStep = 32;   // k per step
    static constexpr int kSub = 2;     // fragment reads per step (16 k each)
    using Frag = f32x4;                // 4 k of one row
    static __device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[v], b[v], c, 0, 0, 0);
        return c;
    }
};
template <>
struct Traits<__bf16> {
    static constexpr int kStep = 64;
    static constexpr int kSub = 2;     // 32 k each
    using Frag = s16x8;                // 8 k of one row
    static __device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <>
struct Traits<_Float16> {
    static constexpr int kStep = 64;
    static constexpr int kSub = 2;
    using Frag = s16x8;
    static __device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

typedef __attribute__((address_space(3))) void *LdsPtr;

// Swizzle key of row kk of a k-major tile of TR rows, in units of 32 bytes (16-bit) or 64
// (fp32); a 64-row tile has four units of 32 bytes, so its key keeps two bits.
template <typename T, int TR>
__device__ __forceinline__ int kmajor_key(int kk) {
    if constexpr (sizeof(T) == 2)
        return ((kk & 3) | ((kk >> 3 & 1) << 2)) & (TR / 16 - 1);
    return kk >> 2 & 3;
}

// The per-thread part of an operand's tile loads: TR rows by one step, NT threads.  TERMS = 2:
// steps from `half` on are those of the high term (an operand of one term has them twice).
template <typename T, bool KM, int TR, int NT, int TERMS = 1>
struct TileLoader {
    static constexpr int kChunks = TR * (kStepBytes / 16);  // 16-byte chunks of a tile
    static constexpr int kLoads = kChunks / NT;
    static_assert(kChunks % NT == 0, "whole loads per thread");
    static constexpr int kRowChunks = KM ? TR * static_cast<int>(sizeof(T)) / 16 : 8;
    static constexpr int kStep = Traits<T>::kStep;

    const char *base;       // first byte of the tile at step 0
    int64_t left;           // bytes from base to the operand's end
    int64_t step_bytes;     // advance of base per step
    int64_t k;              // valid k
    uint32_t off[kLoads];   // byte offsets of this thread's chunks within the tile
    int kchunk;             // k-contiguous: first k of this thread's chunks within a step
    int half;               // steps of a term
    int64_t low;            // bytes from base to the low term's tile

    __device__ __forceinline__ void init(const Operand<T> &o, int64_t row0, int tid) {
        constexpr int kPer16 = 16 / static_cast<int>(sizeof(T));
        k = o.k;
        half = static_cast<int>((k + kStep - 1) / kStep);
        low = o.low;
        if constexpr (KM) {
            base = reinterpret_cast<const char *>(o.p + row0);
            left = ((o.k - 1) * o.ld + o.rows - row0) * static_cast<int64_t>(sizeof(T));
            step_bytes = o.ld * kStep * static_cast<int64_t>(sizeof(T));
            kchunk = 0;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int q = u * NT + tid;
                const int kk = q / kRowChunks, s = q % kRowChunks;
                // chunks per swizzle unit: 2 (32 bytes) or 4 (64 bytes)
                constexpr int kUnit = sizeof(T) == 2 ? 2 : 4;
                const int c = ((s / kUnit) ^ kmajor_key<T, TR>(kk)) * kUnit + s % kUnit;
                // columns past the operand's rows: an offset past its end (zeros)
                off[u] = row0 + c * kPer16 < o.rows
                             ? static_cast<uint32_t>(kk * o.ld * sizeof(T) + c * 16u)
                             : 0xFFFFFFF0u;
            }
        } else {
            base = reinterpret_cast<const char *>(o.p + row0 * o.ld);
            left = ((o.rows - row0 - 1) * o.ld + o.k) * static_cast<int64_t>(sizeof(T));
            step_bytes = kStepBytes;
            const int r0 = tid / 8, s = tid % 8;
            const int c = s ^ (r0 >> 1 & 7);
            kchunk = c * kPer16;
#pragma unroll
            for (int u = 0; u < kLoads; ++u)
                off[u] = static_cast<uint32_t>((r0 + u * (NT / 8)) * o.ld * sizeof(T) + c * 16u);
        }
    }

    // Step s's tile into lds (every wave writes its own 1 KiB pieces).
    __device__ __forceinline__ void load(char *lds, int s, int tid) const {
        const char *from = base;
        if constexpr (TERMS == 2) {
            if (s >= half)
                s -= half;
            else
                from += low;
        }
        const int64_t at = s == kPastEnd ? 0 : s * step_bytes;
        int64_t bytes = s == kPastEnd ? 0 : left - at;
        if (bytes > 0xFFFFFF00ll) bytes = 0xFFFFFF00ll;
        if (bytes < 0) bytes = 0;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(from + at), 0, static_cast<int>(bytes), 0x00020000);
        const bool in = KM || s * static_cast<int64_t>(kStep) + kchunk < k;
        const int wave0 = __builtin_amdgcn_readfirstlane(tid & ~63);
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (LdsPtr)(lds + (u * NT + wave0) * 16), 16,
                static_cast<int>(in ? off[u] : 0xFFFFFFF0u), 0, 0, 0);
    }
};

// Fragment f (16 rows from r0 + 16 f) of sub-step ks: this lane's k values of its row.
template <typename T, bool KM, int TR>
struct FragReader {
    using Frag = typename Traits<T>::Frag;
    int lane;
    int r0;
    __device__ __forceinline__ Frag read(const char *lds, int f, int ks) const {
        const int l16 = lane & 15, g = lane >> 4;
        if constexpr (!KM) {
            const int row = r0 + f * 16 + l16;
            const int slot = (ks * 4 + g) ^ (l16 >> 1 & 7);
            return *reinterpret_cast<const Frag *>(lds + row * 128 + slot * 16);
        } else if constexpr (sizeof(T) == 2) {
            // two transposing reads of 4 k by 16 columns per group of 16 lanes: lane s of
            // the group addresses k row s / 4, columns 4 (s % 4) .. + 3, and receives
            // column s of the four rows
            typedef __attribute__((address_space(3))) s16x4 *P;
            Frag out;
            const int unit = (r0 >> 4) + f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kk = ks * 32 + g * 8 + h * 4 + (l16 >> 2);
                const char *p = lds + kk * (TR * 2) + (unit ^ kmajor_key<T, TR>(kk)) * 32 +
                                (l16 & 3) * 8;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
#pragma unroll
                for (int v = 0; v < 4; ++v) out[h * 4 + v] = t[v];
            }
            return out;
        } else {
            Frag out;
            const int unit = (r0 >> 4) + f;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int kk = ks * 16 + g * 4 + v;
                out[v] = *reinterpret_cast<const float *>(
                    lds + kk * (TR * 4) + (unit ^ kmajor_key<T, TR>(kk)) * 64 + l16 * 4);
            }
            return out;
        }
    }
};

// Tile (ti, tj) of workgroup `wg` of an ni x nj grid of tiles.  Workgroups go round the 8
// XCDs; each XCD gets one contiguous run of the tile order, and that order takes i tiles
// in groups of 8 per j, so that the tiles an XCD has in flight share operand rows in its L2.
__device__ __forceinline__ void tile_of(uint32_t wg, uint32_t ni, uint32_t nj, uint32_t &ti,
                                        uint32_t &tj) {
    constexpr uint32_t kXcds = 8, kGroup = 8;
    const uint32_t n = ni * nj;
    const uint32_t q = n / kXcds, r = n % kXcds, x = wg % kXcds;
    const uint32_t t = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + wg / kXcds;
    const uint32_t per = kGroup * nj;
    const uint32_t first = t / per * kGroup;
    const uint32_t rows = ni - first < kGroup ? ni - first : kGroup;
    const uint32_t in = t % per;
    ti = first + in % rows;
    tj = in / rows;
}

// Waits until at most LOADS of this wave's loads are in flight and its LDS accesses are
// done, then meets the workgroup; no memory access moves across.
template <int LOADS>
__device__ __forceinline__ void meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
}

// The tile's stages in LDS, each a variable of its own.  kRing: five pieces, one operand's
// tile each, that hold A(0) B(0) A(1) B(1) A(2) and go round: tile n is in piece n % 5.
constexpr int kRing = 5;
template <int NB>
struct Stages {
    char *a[NB];
    char *b[NB];
};
template <>
struct Stages<kRing> {
    char *p[kRing];
    // (the pieces of the outputs)
    char *a[1];
};

// Hands out a wave's sums.  16 rows at a time go through a piece of LDS of the wave's own (in a
// stage, which is done with), so that a lane takes four consecutive j of always the same
// column group and a row leaves in one run.  The 16-byte chunks of row r are permuted by r:
// the 16 rows of a fragment otherwise start in the same bank.
template <int FI, int FJ, typename Epi>
__device__ __forceinline__ void hand_out(const f32x4 (&acc)[FI][FJ], char *piece, int lane,
                                         int64_t i0, int64_t j0, const Epi &epi) {
    constexpr int kRow = FJ * 4;  // 16-byte chunks of a row
    static_assert(64 % kRow == 0, "whole rows per wave and turn");
    const int l16 = lane & 15, g = lane >> 4;
    const int rr = lane / kRow, rc = lane % kRow;
    typename Epi::Column col(epi, j0 + rc * 4);
#pragma unroll
    for (int i = 0; i < FI; ++i) {
#pragma unroll
        for (int f = 0; f < FJ; ++f)
            *reinterpret_cast<f32x4 *>(piece + l16 * (FJ * 64) +
                                       (((f * 4 + g) ^ l16) % kRow) * 16) = acc[i][f];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int r = rr; r < 16; r += 64 / kRow) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(piece + r * (FJ * 64) +
                                                             ((rc ^ r) % kRow) * 16);
            epi.put(col, i0 + i * 16 + r, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Computes the tile's sums over steps s_begin .. s_end - 1 and hands it out in pieces of
// four: Epi::Column col(epi, j) once per lane, then epi.put(col, i, D[i][j .. j + 3]) for its
// rows; i and j may lie past I or J.
template <typename T, bool AKM, bool BKM, int TI, int TJ, int WI, int WJ, int NB, int TERMS,
          typename Epi>
__device__ __forceinline__ void gemm_tile(const Operand<T> &A, const Operand<T> &B, int64_t i0,
                                          int64_t j0, int s_begin, int s_end,
                                          const Stages<NB> &st, const Epi &epi) {
    constexpr int NT = WI * WJ * 64;
    constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;
    constexpr int kSub = Traits<T>::kSub;
    using Frag = typename Traits<T>::Frag;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave / WJ, wj = wave % WJ;
    TileLoader<T, AKM, TI, NT, TERMS> la;
    TileLoader<T, BKM, TJ, NT, TERMS> lb;
    la.init(A, i0, tid);
    lb.init(B, j0, tid);
    const FragReader<T, AKM, TI> ra{lane, wi * FI * 16};
    const FragReader<T, BKM, TJ> rb{lane, wj * FJ * 16};
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A step is kSub sub-steps of two phases, each half of the wave's rows i against all its
    // columns j.  A phase first requests the next phase's fragments, then multiplies its
    // own.  Before the last phase all waves meet: every fragment of this step is in
    // registers then, so its stage is refilled (step s + NB), and the next step's first
    // fragments are read while the last phase multiplies.
    constexpr int FH = FI / 2;
    constexpr int kPhases = 2 * kSub;
    static_assert(FI % 2 == 0, "two phases per sub-step");
    Frag fa[2][FH], fb[2][FJ];
    auto read_phase = [&](const char *ta, const char *tb, int ph) {
        const int ks = ph / 2, half = ph % 2;
        if (half == 0) {
#pragma unroll
            for (int j = 0; j < FJ; ++j) fb[ks % 2][j] = rb.read(tb, j, ks);
        }
#pragma unroll
        for (int i = 0; i < FH; ++i) fa[ph % 2][i] = ra.read(ta, half * FH + i, ks);
    };
    auto mul_phase = [&](int ph) {
        const int ks = ph / 2, half = ph % 2;
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j)
                acc[half * FH + i][j] =
                    Traits<T>::mma(fb[ks % 2][j], fa[ph % 2][i], acc[half * FH + i][j]);
    };
    constexpr int kLoadsA = decltype(la)::kLoads, kLoadsB = decltype(lb)::kLoads;
    // (a step past s_end loads nothing that is there)
    auto valid = [&](int s) { return s < s_end ? s : kPastEnd; };
    // Two terms: the sums of the low one are scaled before the high one's first step, or at the
    // end where this tile's steps do not reach it.
    constexpr bool kScaled = TERMS == 2 && kLowShift<T> != 0;
    const int scale_at = kScaled && la.half < s_end ? la.half : kPastEnd;
    auto scale_low = [&] {
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] *= 1.0f / (1 << kLowShift<T>);
    };
    if constexpr (NB == kRing) {
        // Two whole steps of a 256 x 256 tile take 128 of the 160 KiB of LDS, and with two
        // stages every load has one step to arrive.  Five pieces give A two steps: B(s + 2)
        // goes into A(s)'s piece after the meeting of step s, A(s + 3) into B(s)'s in the
        // first phase of step s + 1, so the loads are also spread (8192 x 4096 x 14336 in
        // bf16: 815 us with two stages, 760 with the ring).
        auto step = [&](int s, auto turn) {
            constexpr int t = 2 * decltype(turn)::value;
            char *sa = st.p[t % 5], *sb = st.p[(t + 1) % 5];
            const char *na = st.p[(t + 2) % 5], *nb = st.p[(t + 3) % 5];
            la.load(st.p[(t + 4) % 5], valid(s + 2), tid);
            if constexpr (kScaled)
                if (s == scale_at) scale_low();
#pragma unroll
            for (int ph = 0; ph + 1 < kPhases; ++ph) {
                read_phase(sa, sb, ph + 1);
                mul_phase(ph);
                __builtin_amdgcn_sched_barrier(0);
            }
            meet<kLoadsA>();
            lb.load(sa, valid(s + 2), tid);
            read_phase(na, nb, 0);
            mul_phase(kPhases - 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (s_begin < s_end) {
            la.load(st.p[0], s_begin, tid);
            lb.load(st.p[1], s_begin, tid);
            la.load(st.p[2], valid(s_begin + 1), tid);
            lb.load(st.p[3], valid(s_begin + 1), tid);
            meet<kLoadsA + kLoadsB>();
            read_phase(st.p[0], st.p[1], 0);
            for (int s = s_begin; s < s_end; s += 5) {
                step(s, std::integral_constant<int, 0>{});
                if (s + 1 < s_end) step(s + 1, std::integral_constant<int, 1>{});
                if (s + 2 < s_end) step(s + 2, std::integral_constant<int, 2>{});
                if (s + 3 < s_end) step(s + 3, std::integral_constant<int, 3>{});
                if (s + 4 < s_end) step(s + 4, std::integral_constant<int, 4>{});
            }
            meet<0>();  // no load into LDS outlives the tile
        }
    } else {
        // Step s from (ta, tb); (na, nb) hold step s + 1 from the meeting on.  Steps past
        // s_end multiply zeros.  At a meeting the stages after the next one are in flight.
        auto step = [&](int s, char *ta, char *tb, const char *na, const char *nb) {
            if constexpr (kScaled)
                if (s == scale_at) scale_low();
#pragma unroll
            for (int ph = 0; ph + 1 < kPhases; ++ph) {
                read_phase(ta, tb, ph + 1);
                mul_phase(ph);
                __builtin_amdgcn_sched_barrier(0);
            }
            meet<(NB - 2) * (kLoadsA + kLoadsB)>();
            la.load(ta, valid(s + NB), tid);
            lb.load(tb, valid(s + NB), tid);
            read_phase(na, nb, 0);
            mul_phase(kPhases - 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (s_begin < s_end) {
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                la.load(st.a[t], valid(s_begin + t), tid);
                lb.load(st.b[t], valid(s_begin + t), tid);
            }
            meet<(NB - 1) * (kLoadsA + kLoadsB)>();
            read_phase(st.a[0], st.b[0], 0);
            for (int s = s_begin; s < s_end; s += NB) {
#pragma unroll
                for (int t = 0; t < NB; ++t)
                    step(s + t, st.a[t], st.b[t], st.a[(t + 1) % NB], st.b[(t + 1) % NB]);
            }
            meet<0>();  // no load into LDS outlives the tile
        }
    }
    if constexpr (kScaled)
        if (scale_at == kPastEnd && s_begin < la.half) scale_low();
    static_assert(WI * WJ * FJ * 1024 <= TI * kStepBytes, "the waves' pieces fit the buffer");
    hand_out(acc, st.a[0] + wave * (FJ * 1024), lane, i0 + wi * FI * 16, j0 + wj * FJ * 16, epi);
}

// ---------------------------------------------------------------- fp32 by bf16 terms
//
// The matrix cores multiply bf16 16 times as fast as fp32.  An fp32 number is the sum of three
// bf16 numbers, x = x0 + x1 + x2, and six of the nine products reach fp32's own accuracy:
//     x y ~ x0 y0 + (x0 y1 + x1 y0) + (x1 y1 + x0 y2 + x2 y0).
// x0 is x rounded to nearest, x1 the next eight bits of the rest, x2 what remains (the
// differences are exact).  With 1 <= |x| < 2, |x1| <= 2^-8 and |x2| < 2^-16, so the three left
// out are below (1 + 2^-9) 2^-23 |x y| together, of either sign.  (With x0 truncated they
// reach 2^-7 and 2^-15: 1.96 2^-22 was left out of the square of 1 + 2^-7 - 2^-23, always
// towards zero.  All three rounded: 2^-24, but 4096^3 took 819 us against 808, and 785
// with all truncated.)  Each product is exact and the sums are fp32, in fewer additions than
// the fp32 instruction makes.  (What is below 2^-133, bf16's smallest number, is lost, so numbers
// below 2^-109 keep fewer bits.)  The operands stay fp32 in memory and LDS and are split in registers: about 50 VALU instructions
// for a fragment, which meets FI or FJ others in six matrix instructions each.  VALU issue
// bounds it: 68 % of the clocks at 4096^3 with 64 x 64 per wave, the matrix cores 49 %.  A call
// takes 0.81 ms (170 TFLOP/s); the fp32 instruction took 1.05 (its peak is 157 TFLOP/s), the
// library's product 0.91.
// An infinity has no such split (inf - inf, and inf times a zero term, are NaN), nor has a number
// whose x0 would round to one.  A step that holds an infinity, a NaN or a magnitude from
// (2 - 2^-8) 2^127 on is multiplied both ways, and the outputs whose own row of A or B holds it
// take the fp32 instruction's sums: an output depends on its two rows alone.

struct Terms {
    s16x8 t[3];
};

// Whether any of eight values has no terms.
__device__ __forceinline__ bool has_no_terms(const f32x4 &lo, const f32x4 &hi) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        top = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(__builtin_fabsf(lo[k]), __builtin_fabsf(hi[k])), top);
    return !(top < 0x1.FFp127f);
}

// The terms of eight values.
__device__ __forceinline__ void split_terms(const f32x4 &lo, const f32x4 &hi, Terms &out) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = lo[k];
        x[4 + k] = hi[k];
    }
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 p[3];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const uint32_t b = __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2{x[k], x[k + 1]}), bf16x2));
        p[0][k / 2] = b;
        uint32_t u[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // the differences are exact, and the last has eight bits
            const float r = x[k + e] - __uint_as_float(e ? b & 0xFFFF0000u : b << 16);
            u[e][0] = __float_as_uint(r);
            u[e][1] = __float_as_uint(r - __uint_as_float(u[e][0] & 0xFFFF0000u));
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)  // the upper halves of the pair
            p[1 + t][k / 2] = __builtin_amdgcn_perm(u[1][t], u[0][t], 0x07060302u);
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) out.t[t] = __builtin_bit_cast(s16x8, p[t]);
}

// gemm_tile for fp32 operands, two stages, k in 32s.
template <bool AKM, bool BKM, int TI, int TJ, int WI, int WJ, typename Epi>
__device__ __forceinline__ void gemm_tile_f32(const Operand<float> &A, const Operand<float> &B,
                                              int64_t i0, int64_t j0, int s_begin, int s_end,
                                              const Stages<2> &st, const Epi &epi) {
    constexpr int NT = WI * WJ * 64;
    constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;
    constexpr int FH = FI / 2;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave / WJ, wj = wave % WJ;
    TileLoader<float, AKM, TI, NT> la;
    TileLoader<float, BKM, TJ, NT> lb;
    la.init(A, i0, tid);
    lb.init(B, j0, tid);
    constexpr int kLoads = decltype(la)::kLoads + decltype(lb)::kLoads;
    const FragReader<float, AKM, TI> ra{lane, wi * FI * 16};
    const FragReader<float, BKM, TJ> rb{lane, wj * FJ * 16};
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 xa[FH][2], xb[FJ][2];  // values of the phase to come
    auto read_a = [&](const char *ta, int half) {
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) xa[i][ks] = ra.read(ta, half * FH + i, ks);
    };
    auto read_b = [&](const char *tb) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) xb[j][ks] = rb.read(tb, j, ks);
    };
    Terms pa[FH], pb[FJ];
    // Half the wave's rows against all its columns; k value 4 g + v of either 16 is lane
    // group g's, for both operands.
    auto mul_half = [&](int half) {
        auto mac = [&](int s, int t) {
#pragma unroll
            for (int i = 0; i < FH; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j)
                    acc[half * FH + i][j] =
                        Traits<__bf16>::mma(pb[j].t[s], pa[i].t[t], acc[half * FH + i][j]);
        };
        mac(2, 0);
        mac(0, 2);
        mac(1, 1);
        mac(1, 0);
        mac(0, 1);
        mac(0, 0);
    };
    // Bit r: row r of a fragment has a value without terms (its 32 k are in four lanes).
    auto wild_rows = [&](const f32x4 &lo, const f32x4 &hi) {
        uint64_t m = __ballot(has_no_terms(lo, hi));
        m |= m >> 32;
        m |= m >> 16;
        return static_cast<uint32_t>(m) & 0xFFFFu;
    };
    // Rows with such a value: their outputs take the fp32 instruction's sums, from the tile in
    // LDS, and zeros replace the values to be split.  A lane's four outputs are row l16 of
    // A with rows 4 g .. 4 g + 3 of B.
    auto mul_wild = [&](const char *ta, const char *tb, int half) {
#pragma unroll
        for (int i = 0; i < FH; ++i) {
            const f32x4 a0 = ra.read(ta, half * FH + i, 0), a1 = ra.read(ta, half * FH + i, 1);
            const bool wild_a = wild_rows(a0, a1) >> (lane & 15) & 1;
            if (wild_a) xa[i][0] = xa[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                const f32x4 b0 = rb.read(tb, j, 0), b1 = rb.read(tb, j, 1);
                const uint32_t rows = wild_rows(b0, b1);
                if (half == 0 && i == 0 && (rows >> (lane & 15) & 1))
                    xb[j][0] = xb[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
                const uint32_t wild_b = rows >> (lane >> 4) * 4;
                const f32x4 f = Traits<float>::mma(
                    b1, a1, Traits<float>::mma(b0, a0, f32x4{0.f, 0.f, 0.f, 0.f}));
                f32x4 &c = acc[half * FH + i][j];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (wild_a || (wild_b >> v & 1)) c[v] += f[v];
                __builtin_amdgcn_sched_barrier(0);  // (one at a time: this path's registers)
            }
        }
    };
    auto step = [&](int s, char *ta, char *tb, const char *na, const char *nb) {
        bool wild_b = false;
#pragma unroll
        for (int j = 0; j < FJ; ++j) wild_b |= has_no_terms(xb[j][0], xb[j][1]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            bool wild = wild_b;
#pragma unroll
            for (int i = 0; i < FH; ++i) wild |= has_no_terms(xa[i][0], xa[i][1]);
            if (__builtin_expect(__any(wild), 0)) mul_wild(ta, tb, half);
            if (half == 0) {
#pragma unroll
                for (int j = 0; j < FJ; ++j) split_terms(xb[j][0], xb[j][1], pb[j]);
            }
#pragma unroll
            for (int i = 0; i < FH; ++i) split_terms(xa[i][0], xa[i][1], pa[i]);
            if (half == 0) {
                read_a(ta, 1);
            } else {
                meet<0>();
                la.load(ta, s + 2 < s_end ? s + 2 : kPastEnd, tid);
                lb.load(tb, s + 2 < s_end ? s + 2 : kPastEnd, tid);
                read_a(na, 0);
                read_b(nb);
            }
            mul_half(half);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (s_begin < s_end) {
        la.load(st.a[0], s_begin, tid);
        lb.load(st.b[0], s_begin, tid);
        la.load(st.a[1], s_begin + 1 < s_end ? s_begin + 1 : kPastEnd, tid);
        lb.load(st.b[1], s_begin + 1 < s_end ? s_begin + 1 : kPastEnd, tid);
        meet<kLoads>();
        read_a(st.a[0], 0);
        read_b(st.b[0]);
        for (int s = s_begin; s < s_end; s += 2) {
            step(s, st.a[0], st.b[0], st.a[1], st.b[1]);
            step(s + 1, st.a[1], st.b[1], st.a[0], st.b[0]);
        }
        meet<0>();  // no load into LDS outlives the tile
    }
    static_assert(WI * WJ * FJ * 1024 <= TI * kStepBytes, "the waves' pieces fit the buffer");
    hand_out(acc, st.a[0] + wave * (FJ * 1024), lane, i0 + wi * FI * 16, j0 + wj * FJ * 16, epi);
}

}  // namespace gemm
}  // namespace tcq
