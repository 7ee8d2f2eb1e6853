// The microscaled linear layer: y = xq W^T + bias + residual for a matrix W of 4-bit codes and
// rows xq quantised to 4 or 8 bits, and its gradients.
//
// A product of two E2M1 codes is a multiple of 1/4 below 37, so the matrix instruction that
// takes both operands as codes with their scale bytes adds a group's 32 products exactly, and the
// groups in fp32.  Its E4M3 form does not: it aligns eight products to the largest and drops
// what lies 2^-13 below (256 + 2^-6 gives 256), so 8-bit rows are multiplied as bf16 numbers,
// which hold every code times its scale, with exact products and fp32 sums.
#include <hip/hip_runtime.h>

#include "gemm_device.h"
#include "linear_epilogue.h"
#include "mx_unpack_device.h"
#include "tcq.h"
#include "tcq_internal.h"

namespace tcq {
namespace gemm {

// Two 4-bit codes: k is counted in bytes, 128 to a step (two instructions of 128 codes).
struct CodePair {
    uint8_t b;
};
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

}  // namespace gemm

namespace {

using gemm::CodePair;
using gemm::i32x4;
using gemm::i32x8;
using gemm::Operand;
using gemm::s16x8;

__device__ __forceinline__ i32x8 wide(const i32x4 &v) {
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// c += codes of a and b, a's scale in byte OA of sa and b's in byte OB of sb (16 rows of 128
// codes each: lane l holds group l / 16 of row l % 16 of either, and the group's scale).
template <int OA, int OB>
__device__ __forceinline__ f32x4 mma_fp4(const i32x4 &a, uint32_t sa, const i32x4 &b, uint32_t sb,
                                         const f32x4 &c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a), wide(b), c, 4, 4, OA,
                                                            static_cast<int>(sa), OB,
                                                            static_cast<int>(sb));
}
// The same for bytes known once the loops around are unrolled.
__device__ __forceinline__ f32x4 mma_fp4_at(int oa, int ob, const i32x4 &a, uint32_t sa,
                                            const i32x4 &b, uint32_t sb, const f32x4 &c) {
    switch (oa * 4 + ob) {
#define TCQ_AT(A, B) \
    case A * 4 + B: return mma_fp4<A, B>(a, sa, b, sb, c);
#define TCQ_ROW(A) TCQ_AT(A, 0) TCQ_AT(A, 1) TCQ_AT(A, 2) TCQ_AT(A, 3)
        TCQ_ROW(0) TCQ_ROW(1) TCQ_ROW(2) TCQ_ROW(3)
#undef TCQ_ROW
#undef TCQ_AT
    }
    return c;
}

// ---------------------------------------------------------------- large batches, 4-bit rows

// Scale bytes in the order in which the product's lanes take them: 128 rows by one step (eight
// groups) are 1 KiB, lane l's 16 bytes at 16 l hold, for row 16 f + l % 16 of the tile, f = 0
// .. 7, groups l / 16 and 4 + l / 16 of the step in bytes 2 f and 2 f + 1.  So a wave reads
// a step's scales in one contiguous access per operand.  Rows and groups past the end get 1.
//   A thread takes a step of the eight rows l16, 16 + l16, ..: eight bytes of each, four pieces out
// (6.6 us for the 12288 rows of 8192 x 4096 x 14336).
struct ScaleArgs {
    const uint8_t *scale;
    int64_t rows, groups;
    uint32_t steps;
    uint8_t *out;
    int64_t work;    // tiles x 16 x steps
};
__device__ __forceinline__ void order_scales(const ScaleArgs &a, int64_t q) {
    const int64_t tl = q / a.steps;
    const uint32_t step = static_cast<uint32_t>(q - tl * a.steps);
    const int64_t tile = tl >> 4, row0 = tile * 128 + (tl & 15);
    const int64_t g0 = static_cast<int64_t>(step) * 8;
    uint32_t w[4][4];
    struct __attribute__((packed)) Eight { uint32_t v[2]; };
    Eight e[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) {
        const int64_t row = row0 + 16 * f;
        e[f].v[0] = e[f].v[1] = 0x7F7F7F7Fu;
        if (row < a.rows) {
            const uint8_t *p = a.scale + row * a.groups + g0;
            if (g0 + 8 <= a.groups) {
                e[f] = *reinterpret_cast<const Eight *>(p);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (g0 + k < a.groups)
                        e[f].v[k / 4] = (e[f].v[k / 4] & ~(255u << (8 * (k % 4)))) |
                                        static_cast<uint32_t>(p[k]) << (8 * (k % 4));
            }
        }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int f = 0; f < 8; f += 2)
            w[g][f / 2] = (e[f].v[0] >> (8 * g) & 255u) | (e[f].v[1] >> (8 * g) & 255u) << 8 |
                          (e[f + 1].v[0] >> (8 * g) & 255u) << 16 |
                          (e[f + 1].v[1] >> (8 * g) & 255u) << 24;
    uint4 *out = reinterpret_cast<uint4 *>(a.out) + (tile * a.steps + step) * 64 + (tl & 15);
#pragma unroll
    for (int g = 0; g < 4; ++g) out[g * 16] = make_uint4(w[g][0], w[g][1], w[g][2], w[g][3]);
}
__global__ __launch_bounds__(256) void order_scales_kernel(ScaleArgs x, ScaleArgs w) {
    const int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (q < x.work)
        order_scales(x, q);
    else if (q - x.work < w.work)
        order_scales(w, q - x.work);
}

// The ordered scales of F fragments (16 rows each) of one operand, from row r0 on: a uniform
// address and the lane's offset.
template <int F>
struct ScaleReader {
    static constexpr int kWords = F / 2;
    const uint8_t *base;
    uint32_t off;
    __device__ __forceinline__ ScaleReader(const uint8_t *scales, int64_t r0, int64_t steps,
                                           int lane)
        : base(scales + (r0 / 128) * steps * 1024 + (r0 % 128) / 8), off(lane * 16) {}
    __device__ __forceinline__ void read(int s, uint32_t (&w)[kWords]) const {
        const uint8_t *p = base + s * int64_t{1024};
        if constexpr (kWords == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + off);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p + off);
            w[0] = v.x, w[1] = v.y;
        }
    }
};

// The loads of a tile of TR rows by one step, as TileLoader's (chunk c of row r into slot c ^ (r >>
// 1 & 7), zeros past the rows and past k), with one offset of 32 bits per thread (rows at most
// kMostPitch bytes apart): a thread's rows lie NT / 8 rows apart.  `renew` makes an offset a new
// value to the compiler, which otherwise holds every sum with it in registers, 26 of them, and
// spills to make room; a spill's return waits for all loads on their way.
template <int TR, int NT>
struct CodeLoader {
    static constexpr int kLoads = TR * 8 / NT;
    const char *base;     // uniform, as all but off and chunk
    int64_t left;
    uint32_t apart;
    int k;
    uint32_t off;
    int chunk;            // this thread's first byte within a step
    __device__ __forceinline__ CodeLoader(const Operand<CodePair> &o, int64_t row0, int tid) {
        base = reinterpret_cast<const char *>(o.p + row0 * o.ld);
        left = (o.rows - row0 - 1) * o.ld + o.k;
        apart = static_cast<uint32_t>(NT / 8 * o.ld);
        k = static_cast<int>(o.k);
        const int r = tid / 8;
        chunk = (tid % 8 ^ (r >> 1 & 7)) * 16;
        off = static_cast<uint32_t>(r * o.ld) + chunk;
    }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(off)); }
    // Step s, or zeros from s_end on.  (No branch: matrix instructions would be moved past it, away
    // from the reads that feed them.)
    __device__ __forceinline__ void load(char *lds, int s, int s_end, int tid) const {
        const int64_t at = s * int64_t{gemm::kStepBytes}, rest = left - at;
        const uint32_t most = rest < 0xFFFFFF00ll ? static_cast<uint32_t>(rest) : 0xFFFFFF00u;
        const uint32_t bytes = s < s_end ? most : 0u;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(base + at), 0, static_cast<int>(bytes), 0x00020000);
        const bool in = chunk < k - static_cast<int>(at);
        const int wave0 = __builtin_amdgcn_readfirstlane(tid & ~63);
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (gemm::LdsPtr)(lds + (u * NT + wave0) * 16), 16,
                static_cast<int>(in ? off + u * apart : 0xFFFFFFF0u), 0, 0, 0);
    }
};

// Reads fragments of a tile as FragReader does, from one offset per lane: the slots of the two
// halves of a step differ by an exclusive or with 64.
struct SlotReader {
    int at;
    __device__ __forceinline__ SlotReader(int lane, int r0)
        : at((r0 + (lane & 15)) * 128 + ((lane >> 4) ^ (lane >> 1 & 7)) * 16) {}
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(at)); }
    __device__ __forceinline__ i32x4 read(const char *lds, int f, int ks) const {
        return *reinterpret_cast<const i32x4 *>(lds + (at ^ (ks * 64)) + f * 2048);
    }
};

// A TI x TJ tile of A B^T over the steps s_begin .. s_end - 1 of 256 codes, as gemm_tile's (loads
// straight into LDS, NB stages or a ring of five pieces, phases of some of a wave's rows), with
// the scales of the step to come read from memory into registers.
template <int TI, int TJ, int WI, int WJ, int NB, typename Epi>
__device__ __forceinline__ void mx_tile(const Operand<CodePair> &A, const uint8_t *as,
                                        const Operand<CodePair> &B, const uint8_t *bs,
                                        int64_t steps, int64_t i0, int64_t j0, int s_begin,
                                        int s_end, const gemm::Stages<NB> &st, const Epi &epi) {
    constexpr int NT = WI * WJ * 64;
    constexpr int FI = TI / WI / 16, FJ = TJ / WJ / 16;
    // fragments of A to a phase (two to a phase of 256 rows: 8192 x 4096 x 14336 224.9 us, four
    // 223.2)
    constexpr int FH = FI / 2, kParts = FI / FH, kPhases = 2 * kParts;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave / WJ, wj = wave % WJ;
    CodeLoader<TI, NT> la(A, i0, tid);
    CodeLoader<TJ, NT> lb(B, j0, tid);
    SlotReader ra(lane, wi * FI * 16), rb(lane, wj * FJ * 16);
    const ScaleReader<FI> rsa(as, i0 + wi * FI * 16, steps, lane);
    const ScaleReader<FJ> rsb(bs, j0 + wj * FJ * 16, steps, lane);
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    i32x4 fa[2][FH], fb[2][FJ];
    uint32_t sa[FI / 2], sb[FJ / 2], na_s[FI / 2], nb_s[FJ / 2];
    auto read_phase = [&](const char *ta, const char *tb, int ph) {
        const int ks = ph / kParts, part = ph % kParts;
        if (part == 0) {
#pragma unroll
            for (int j = 0; j < FJ; ++j) fb[ks % 2][j] = rb.read(tb, j, ks);
        }
#pragma unroll
        for (int i = 0; i < FH; ++i) fa[ph % 2][i] = ra.read(ta, part * FH + i, ks);
    };
    auto mul_phase = [&](int ph) {
        const int ks = ph / kParts, part = ph % kParts;
#pragma unroll
        for (int i = 0; i < FH; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                const int fi = part * FH + i;
                f32x4 &c = acc[fi][j];
                c = mma_fp4_at(2 * (j % 2) + ks, 2 * (fi % 2) + ks, fb[ks % 2][j], sb[j / 2],
                               fa[ph % 2][i], sa[fi / 2], c);
            }
    };
    constexpr int kLoadsA = decltype(la)::kLoads, kLoadsB = decltype(lb)::kLoads;
    auto clamped = [&](int s) { return s < s_end ? s : s_end - 1; };
    auto next_scales = [&](int s) {
        rsa.read(clamped(s), na_s);
        rsb.read(clamped(s), nb_s);
    };
    auto take_scales = [&] {
#pragma unroll
        for (int i = 0; i < FI / 2; ++i) sa[i] = na_s[i];
#pragma unroll
        for (int j = 0; j < FJ / 2; ++j) sb[j] = nb_s[j];
    };
    if (s_begin < s_end) {
        next_scales(s_begin);
        if constexpr (NB == gemm::kRing) {
            auto step = [&](int s, auto turn) {
                constexpr int t = 2 * decltype(turn)::value;
                char *ta = st.p[t % 5], *tb = st.p[(t + 1) % 5];
                const char *na = st.p[(t + 2) % 5], *nb = st.p[(t + 3) % 5];
                take_scales();
                next_scales(s + 1);
                ra.renew();
                rb.renew();
                la.renew();
                lb.renew();
                la.load(st.p[(t + 4) % 5], s + 2, s_end, tid);
#pragma unroll
                for (int ph = 0; ph + 1 < kPhases; ++ph) {
                    read_phase(ta, tb, ph + 1);
                    mul_phase(ph);
                    __builtin_amdgcn_sched_barrier(0);
                }
                gemm::meet<kLoadsA>();
                lb.load(ta, s + 2, s_end, tid);
                read_phase(na, nb, 0);
                mul_phase(kPhases - 1);
                __builtin_amdgcn_sched_barrier(0);
            };
            la.load(st.p[0], s_begin, s_end, tid);
            lb.load(st.p[1], s_begin, s_end, tid);
            la.load(st.p[2], s_begin + 1, s_end, tid);
            lb.load(st.p[3], s_begin + 1, s_end, tid);
            gemm::meet<kLoadsA + kLoadsB>();
            read_phase(st.p[0], st.p[1], 0);
            for (int s = s_begin;;) {
                step(s, std::integral_constant<int, 0>{});
                if (++s == s_end) break;
                step(s, std::integral_constant<int, 1>{});
                if (++s == s_end) break;
                step(s, std::integral_constant<int, 2>{});
                if (++s == s_end) break;
                step(s, std::integral_constant<int, 3>{});
                if (++s == s_end) break;
                step(s, std::integral_constant<int, 4>{});
                if (++s == s_end) break;
            }
        } else {
            auto step = [&](int s, char *ta, char *tb, const char *na, const char *nb) {
                take_scales();
                next_scales(s + 1);
                ra.renew();
                rb.renew();
                la.renew();
                lb.renew();
#pragma unroll
                for (int ph = 0; ph + 1 < kPhases; ++ph) {
                    read_phase(ta, tb, ph + 1);
                    mul_phase(ph);
                    __builtin_amdgcn_sched_barrier(0);
                }
                gemm::meet<(NB - 2) * (kLoadsA + kLoadsB)>();
                la.load(ta, s + NB, s_end, tid);
                lb.load(tb, s + NB, s_end, tid);
                read_phase(na, nb, 0);
                mul_phase(kPhases - 1);
                __builtin_amdgcn_sched_barrier(0);
            };
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                la.load(st.a[t], s_begin + t, s_end, tid);
                lb.load(st.b[t], s_begin + t, s_end, tid);
            }
            gemm::meet<(NB - 1) * (kLoadsA + kLoadsB)>();
            read_phase(st.a[0], st.b[0], 0);
            for (int s = s_begin; s < s_end; s += NB) {
#pragma unroll
                for (int t = 0; t < NB; ++t)
                    step(s + t, st.a[t], st.b[t], st.a[(t + 1) % NB], st.b[(t + 1) % NB]);
            }
        }
        gemm::meet<0>();  // no load into LDS outlives the tile
    }
    static_assert(WI * WJ * FJ * 1024 <= TI * gemm::kStepBytes, "the waves' pieces fit the buffer");
    gemm::hand_out(acc, st.a[0] + wave * (FJ * 1024), lane, i0 + wi * FI * 16, j0 + wj * FJ * 16,
                   epi);
}

// A step is 256 columns: 128 bytes of each row's codes, which go into LDS as they are, and two
// matrix instructions deep.  256 x 256 tiles: eight waves of 128 x 64 and a ring of five half
// stages, one step on its way beside the two that are multiplied; 128 x 128: four waves of 64 x 64
// and four stages.  The phase before a meeting reads the next step's first fragments, and loads and
// branches are kept out of the instructions' way.
//   8192 x 4096 x 14336: 226 us, 4.3 PF (a library's product of the same type 291 us).  The matrix
// cores are busy for 42 % of the clocks under the profiler, LDS for 17, and the waves wait for 40 %
// of their time, for a step's loads and meeting.  (Other phases, no order of reads and products,
// and a raised wave priority around the products: all within 1 %.)
template <int TI, int TJ, int WI, int WJ, int NB, typename Epi>
__global__ __launch_bounds__(WI *WJ * 64) void mx_gemm_kernel(Operand<CodePair> A,
                                                              const uint8_t *as,
                                                              Operand<CodePair> B,
                                                              const uint8_t *bs, int steps,
                                                              int steps_per_split, Epi epi,
                                                              uint32_t ni, uint32_t nj) {
    static_assert(NB == 4 || NB == gemm::kRing, "stages");
    __shared__ __align__(16) char a0[TI * gemm::kStepBytes];
    __shared__ __align__(16) char a1[TI * gemm::kStepBytes];
    __shared__ __align__(16) char a2[TI * gemm::kStepBytes];
    __shared__ __align__(16) char b0[TJ * gemm::kStepBytes];
    __shared__ __align__(16) char b1[TJ * gemm::kStepBytes];
    gemm::Stages<NB> st;
    st.a[0] = a0;
    if constexpr (NB == gemm::kRing) {
        static_assert(TI == TJ, "pieces of one size");
        st.p[0] = a0, st.p[1] = b0, st.p[2] = a1, st.p[3] = b1, st.p[4] = a2;
    } else {
        __shared__ __align__(16) char a3[TI * gemm::kStepBytes];
        __shared__ __align__(16) char b2[TJ * gemm::kStepBytes];
        __shared__ __align__(16) char b3[TJ * gemm::kStepBytes];
        st.a[1] = a1, st.a[2] = a2, st.a[3] = a3;
        st.b[0] = b0, st.b[1] = b1, st.b[2] = b2, st.b[3] = b3;
    }
    uint32_t ti, tj;
    gemm::tile_of(blockIdx.x, ni, nj, ti, tj);
    const int s0 = blockIdx.y * steps_per_split;
    const int s1 = s0 + steps_per_split < steps ? s0 + steps_per_split : steps;
    if constexpr (__is_same(Epi, PartEpilogue))
        epi.part += static_cast<int64_t>(blockIdx.y) * epi.I * epi.ld;
    mx_tile<TI, TJ, WI, WJ, NB>(A, as, B, bs, steps, static_cast<int64_t>(ti) * TI,
                                static_cast<int64_t>(tj) * TJ, s0, s1, st, epi);
}

// ---------------------------------------------------------------- few rows of x

// y for 16 BT rows of x (blockIdx.y's).  A workgroup of eight waves takes 16 rows of W at a time;
// the waves share their columns in pairs of 128 (eight groups).  W is read once, straight into the
// matrix instruction's operand: lane (l16, g) reads groups 2 g and 2 g + 1 of a pair, 32 bytes of
// row l16, so that an instruction touches a line of each row and the two scales are one access.
// With 4-bit rows the codes are the operand; with 8-bit ones a group's 32 codes become four bf16
// fragments, fragment j holding columns 8 j .. 8 j + 7 of the lane's group.  Either is another
// order of k than memory's, the same for both operands.
//   The next chunk's W, or the next rows', is on its way while one is multiplied and the waves'
// sums meet in LDS (in wave order, in two halves by turns).
//   DENSE: x comes as it is (few values) and is quantised into LDS by every workgroup, in the
// form the products read.  Otherwise it comes in the order in which the lanes read it (one
// contiguous KiB per instruction: 16 rows of codes as they lie cost an instruction 16 lines).
//   Bound by memory and its first answer: 1 x 14336 x 4096 with 8-bit rows 10.4 us (3.0 TB/s of W),
// of which a launch that only ends takes 2; 100 x 4096 x 4096 with 4-bit rows 7.8, bound by reading
// the rows again in all 256 workgroups.
constexpr int kMxWaves = 8;

struct MxSmallArgs {
    const uint8_t *w, *ws;
    int64_t ldw;
    int64_t M;
    int N, groups, pairs, tiles;
    const void *x;
    int64_t ldx;
    const uint8_t *xq;       // in order
    const uint16_t *xs;
    int B, nbt, per;         // tiles of 16 rows, in all and to a workgroup (at most BT)
    int ldl;                 // bytes of a row of x in LDS (DENSE)
    int red;                 // where the sums' halves start in LDS
};

template <int FMT>
struct XFragment {
    i32x4 q[FMT == TCQ_FP4 ? 1 : 2];   // a group's codes
};

// Four bf16 fragments of a group of 32 codes.
template <int FMT>
__device__ __forceinline__ void group_bf16(const i32x4 *q, float s, s16x8 (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t o[4];
        if constexpr (FMT == TCQ_FP4) {
            mx::decode_word_bf16<FMT>(static_cast<uint32_t>(q[0][j]), s, o);
        } else {
            mx::decode_word_bf16<FMT>(static_cast<uint32_t>(q[j / 2][2 * (j % 2)]), s, o);
            mx::decode_word_bf16<FMT>(static_cast<uint32_t>(q[j / 2][2 * (j % 2) + 1]), s, o + 2);
        }
        f[j] = __builtin_bit_cast(s16x8,
                                  (i32x4{static_cast<int>(o[0]), static_cast<int>(o[1]),
                                         static_cast<int>(o[2]), static_cast<int>(o[3])}));
    }
}

template <typename T, int FMT, int BT, bool DENSE>
__global__ __launch_bounds__(kMxWaves * 64) void mx_small_kernel(MxSmallArgs a,
                                                                 LayerEpilogue<T> epi) {
    extern __shared__ __align__(16) char lds[];
    constexpr int U = 2;    // pairs of a chunk
    const int tid = threadIdx.x;
    const int lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p0 = wave * a.pairs / kMxWaves, p1 = (wave + 1) * a.pairs / kMxWaves;
    const int chunks = ((a.pairs + kMxWaves - 1) / kMxWaves + U - 1) / U;   // of the longest share
    struct WPair {
        i32x4 q[2];
        uint32_t e;      // two scale bytes
    };
    WPair w[U];
    // Pair p of the tile's rows, or zeros (groups past the end: codes of zero, scales of 1).
    auto load_w = [&](int tile, int p, WPair &o) {
        const int64_t j = static_cast<int64_t>(tile) * 16 + l16;
        const int64_t row = j < a.M ? j : a.M - 1;
        const int grp = p * 8 + 2 * g;
        o.q[0] = o.q[1] = i32x4{0, 0, 0, 0};
        o.e = 0x7F7Fu;
        if (p >= p1 || tile >= a.tiles) return;
        const uint8_t *q = a.w + row * a.ldw + grp * 16, *e = a.ws + row * a.groups + grp;
        if (p * 8 + 8 <= a.groups) {
            struct __attribute__((packed)) Two { uint16_t v; };
            o.q[0] = *reinterpret_cast<const i32x4 *>(q);
            o.q[1] = *reinterpret_cast<const i32x4 *>(q + 16);
            o.e = reinterpret_cast<const Two *>(e)->v;
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (grp + k < a.groups) {
                    o.q[k] = *reinterpret_cast<const i32x4 *>(q + 16 * k);
                    o.e = (o.e & ~(255u << (8 * k))) | static_cast<uint32_t>(e[k]) << (8 * k);
                }
        }
    };
    const int bt0 = blockIdx.y * a.per;    // the first of its tiles of rows
    const int nbt = a.nbt - bt0 < a.per ? a.nbt - bt0 : a.per;
    int tile = blockIdx.x;
#pragma unroll
    for (int k = 0; k < U; ++k) load_w(tile, p0 + k, w[k]);
    char *xscale = lds + a.B * a.ldl;  // (DENSE, 4-bit: scale bytes, pairs x 8 to a row)
    if constexpr (DENSE) {
        // four lanes to a group; groups up to whole pairs
        const int per = a.pairs * 32;
        const T *X = static_cast<const T *>(a.x);
        for (int i = tid; i < a.B * per; i += kMxWaves * 64) {
            const int r = i / per, c = i - r * per;
            const int left = a.N - c * 8;  // may be <= 0
            float v[8];
            if (left >= 8) {
                const Packed<T> p = *reinterpret_cast<const Packed<T> *>(X + r * a.ldx + c * 8);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(p.v[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = k < left ? static_cast<float>(X[r * a.ldx + c * 8 + k]) : 0.0f;
            }
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t m = __float_as_uint(v[k]) & 0x7FFFFFFFu;
                top = top > m ? top : m;
            }
            const int e = mx::scale_byte<FMT>(mx::group_top(top));
            uint32_t q[2];
            mx::encode8<FMT>(v, e, q);
            if constexpr (FMT == TCQ_FP4) {
                *reinterpret_cast<uint32_t *>(lds + r * a.ldl + c * 4) = q[0];
                if ((c & 3) == 0) xscale[r * a.pairs * 8 + (c >> 2)] = static_cast<char>(e);
            } else {
                uint32_t o[4];
                mx::decode_word_bf16<FMT>(q[0], mx::scale_of(e), o);
                mx::decode_word_bf16<FMT>(q[1], mx::scale_of(e), o + 2);
                *reinterpret_cast<uint4 *>(lds + r * a.ldl + c * 16) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        __syncthreads();
    }
    f32x4 acc[BT];
    auto multiply = [&](int p, const WPair &c) {
        if constexpr (DENSE) {
            static_assert(!DENSE || BT == 1, "one tile of rows");
            const int grp = p * 8 + 2 * g;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if constexpr (FMT == TCQ_FP4) {
                    i32x4 xq = {0, 0, 0, 0};
                    uint32_t xe = 127;
                    if (l16 < a.B) {
                        xq = *reinterpret_cast<const i32x4 *>(lds + l16 * a.ldl + (grp + k) * 16);
                        xe = static_cast<uint8_t>(xscale[l16 * a.pairs * 8 + grp + k]);
                    }
                    acc[0] = k == 0 ? mma_fp4<0, 0>(c.q[0], c.e, xq, xe, acc[0])
                                    : mma_fp4<1, 0>(c.q[1], c.e, xq, xe, acc[0]);
                } else {
                    s16x8 wf[4];
                    group_bf16<TCQ_FP4>(&c.q[k], mx::scale_of(c.e >> (8 * k) & 255), wf);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s16x8 xf = {0, 0, 0, 0, 0, 0, 0, 0};
                        if (l16 < a.B)
                            xf = *reinterpret_cast<const s16x8 *>(lds + l16 * a.ldl +
                                                                  (grp + k) * 64 + j * 16);
                        acc[0] = gemm::Traits<__bf16>::mma(wf[j], xf, acc[0]);
                    }
                }
            }
        } else {
            constexpr int kHalves = FMT == TCQ_FP4 ? 1 : 2;
            XFragment<FMT> x[BT][2];
            uint32_t xe[BT];
#pragma unroll
            for (int b = 0; b < BT; ++b) {
                // (tiles of rows past the last repeat it: their sums are not stored)
                const int t = bt0 + (b < nbt ? b : nbt - 1);
                const int64_t at = static_cast<int64_t>(p) * a.nbt + t;
                const i32x4 *q = reinterpret_cast<const i32x4 *>(a.xq) + at * (128 * kHalves) + lane;
                xe[b] = a.xs[at * 64 + lane];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) x[b][k].q[h] = q[(k * kHalves + h) * 64];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                s16x8 wf[4];
                if constexpr (FMT == TCQ_FP8)
                    group_bf16<TCQ_FP4>(&c.q[k], mx::scale_of(c.e >> (8 * k) & 255), wf);
#pragma unroll
                for (int b = 0; b < BT; ++b) {
                    if constexpr (FMT == TCQ_FP4) {
                        acc[b] = k == 0 ? mma_fp4<0, 0>(c.q[0], c.e, x[b][0].q[0], xe[b], acc[b])
                                        : mma_fp4<1, 1>(c.q[1], c.e, x[b][1].q[0], xe[b], acc[b]);
                    } else {
                        s16x8 xf[4];
                        group_bf16<TCQ_FP8>(x[b][k].q, mx::scale_of(xe[b] >> (8 * k) & 255), xf);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[b] = gemm::Traits<__bf16>::mma(wf[j], xf[j], acc[b]);
                    }
                }
            }
        }
    };
    for (int turn = 0; tile < a.tiles; tile += gridDim.x, turn ^= 1) {
#pragma unroll
        for (int b = 0; b < BT; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < chunks; ++c) {
            const bool last = c + 1 == chunks;
            const int next = last ? tile + static_cast<int>(gridDim.x) : tile;
            const int from = last ? p0 : p0 + (c + 1) * U;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const WPair now = w[k];
                load_w(next, from + k, w[k]);
                if (p0 + c * U + k < p1) multiply(p0 + c * U + k, now);
            }
        }
        // The waves' sums: 16 BT x 16 values each, value (row j of W, row b of x) of a tile in word
        // (j / 4 * 16 + b) * 4 + j % 4.
        float *red = reinterpret_cast<float *>(lds + a.red) + turn * (kMxWaves * BT * 256);
#pragma unroll
        for (int b = 0; b < BT; ++b)
            *reinterpret_cast<f32x4 *>(red + ((wave * BT + b) * 64 + lane) * 4) = acc[b];
        __syncthreads();
        for (int i = tid; i < nbt * 256; i += kMxWaves * 64) {
            const int j = i & 15, b = i >> 4;
            const int at = (b >> 4) * 256 + ((j >> 2) * 16 + (b & 15)) * 4 + (j & 3);
            float s = red[at];
#pragma unroll
            for (int v = 1; v < kMxWaves; ++v) s += red[v * BT * 256 + at];
            epi.put_one(bt0 * 16 + b, static_cast<int64_t>(tile) * 16 + j, s);
        }
    }
}

// Codes of B rows as they lie into the order in which mx_small_kernel's lanes read them: pair, tile
// of 16 rows, group of the lane's two, half (8-bit), lane; scales: pair, tile, lane, group.  16
// bytes a thread.
template <int FMT>
__global__ __launch_bounds__(256) void order_rows_kernel(const uint8_t *__restrict__ codes,
                                                         int64_t ld,
                                                         const uint8_t *__restrict__ scale, int B,
                                                         int groups, MxOrder out, int64_t work) {
    constexpr int kHalves = FMT == TCQ_FP4 ? 1 : 2;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < work;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int lane = static_cast<int>(i & 63), h = static_cast<int>((i >> 6) % kHalves);
        const int64_t rest = (i >> 6) / kHalves;
        const int k = static_cast<int>(rest & 1), t = static_cast<int>((rest >> 1) % out.nbt);
        const int64_t p = (rest >> 1) / out.nbt;
        const int r = t * 16 + (lane & 15), grp = static_cast<int>(p) * 8 + 2 * (lane >> 4) + k;
        const bool in = r < B && grp < groups;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in)
            v = *reinterpret_cast<const uint4 *>(codes + r * ld +
                                                 (static_cast<int64_t>(grp) * kHalves + h) * 16);
        reinterpret_cast<uint4 *>(out.codes)[i] = v;
        if (h == 0)
            out.scale[((p * out.nbt + t) * 64 + lane) * 2 + k] =
                in ? scale[static_cast<int64_t>(r) * groups + grp] : 127;
    }
}

// ---------------------------------------------------------------- host side

// Whether mx_small_kernel takes B rows of x; never one batch and not a smaller one (us per call in
// a graph, it / the tiled product).  4-bit rows up to 128, and beyond while a row of W's tiles and
// of x's shares makes at most 896 workgroup turns: 256 x 2048 x 2048 8.7 / 17.3, 384 x 4096 x 4096
// 24.1 / 26.2, 128 x 14336 x 4096 26.6 / 25.7 (with one row more); 512 x 4096 x 4096 31.0 / 27.0.
// 8-bit rows, whose tiled product needs W in 16 bits, up to 512: 160 x 4096 x 4096 23.1 / 37.5, 512
// x 4096 x 4096 44.1 / 44.8, 512 x 14336 x 4096 138 / 161.
bool mx_small(int format, int64_t B, int64_t M) {
    if (format == TCQ_FP8) return B <= 512;
    return B <= 128 || (B + 127) / 128 * ((M + 15) / 16) <= 896;
}

// Values of x that mx_small_kernel quantises by itself, in every workgroup, rather than a launch
// before it (us per call in a graph, it / the two: fp8 1 x 4096 x 4096 5.6 / 7.1, 1 x 4096 x 14336
// 11.7 / 12.9, 4 x 4096 x 4096 6.9 / 6.9, 8 x 4096 x 4096 8.7 / 7.0; fp4 16 x 2048 x 2048 7.4 /
// 6.0).
constexpr int64_t kMxDenseValues = 16384;

// Workgroups of 256 threads, each of which takes every so many-th of `work` pieces.
uint32_t blocks_for(int64_t work) {
    const int64_t n = (work + 255) / 256;
    return static_cast<uint32_t>(n < (1 << 20) ? n : 1 << 20);
}

size_t pad(int64_t n, int64_t to) { return static_cast<size_t>((n + to - 1) / to * to); }

int64_t groups_of(int64_t n) { return (n + mx::kGroup - 1) / mx::kGroup; }

template <typename T>
LayerEpilogue<T> mx_epilogue(const MxLinearCall &c) {
    LayerEpilogue<T> e{};
    e.bias = c.bias;
    e.res = static_cast<const T *>(c.residual);
    e.y = static_cast<T *>(c.y);
    e.ldr = c.ldr;
    e.ldy = c.ldy;
    e.I = c.B;
    e.J = c.M;
    e.act = TCQ_ACT_NONE;
    e.vec_y = four_aligned(e.y, e.ldy);
    e.vec_r = e.res && four_aligned(e.res, e.ldr);
    return e;
}

int64_t pairs_of(int64_t groups) { return (groups + 7) / 8; }

// LDS row of x quantised in the kernel: whole pairs, 16 bytes more so that rows start in
// different banks.
int dense_row(int format, int64_t pairs) {
    return static_cast<int>(pairs * (format == TCQ_FP4 ? 128 : 512) + 16);
}
int64_t dense_bytes(int format, int64_t B, int64_t pairs) {
    return align_up(B * (dense_row(format, pairs) + (format == TCQ_FP4 ? pairs * 8 : 0)), 16);
}
bool small_dense(const MxLinearCall &c) {
    return c.x && !c.keep && c.B <= 16 && c.B * c.N <= kMxDenseValues;
}

template <typename T, int FMT, int BT, bool DENSE>
hipError_t launch_small_as(MxSmallArgs a, const LayerEpilogue<T> &epi, hipStream_t s) {
    // LDS: sums, and x quantised in the kernel, at most 2 kMxDenseValues + 16 x 526 bytes
    constexpr int kSums = 2 * kMxWaves * BT * 1024;
    static_assert(!DENSE || kSums + 2 * kMxDenseValues + 16 * 526 <= 64 << 10, "");
    a.red = DENSE ? static_cast<int>(dense_bytes(FMT, a.B, a.pairs)) : 0;
    if (kSums > 64 << 10) {
        const void *kern = reinterpret_cast<const void *>(mx_small_kernel<T, FMT, BT, DENSE>);
        const hipError_t e =
            hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, kSums);
        if (e != hipSuccess) return e;
    }
    // as many rounds of tiles for every workgroup
    const int64_t most = (BT == 1 ? 2 : 1) * 256, rounds = (a.tiles + most - 1) / most;
    const int64_t grid = (a.tiles + rounds - 1) / rounds;
    const unsigned shares = static_cast<unsigned>((a.nbt + a.per - 1) / a.per);
    hipLaunchKernelGGL((mx_small_kernel<T, FMT, BT, DENSE>),
                       dim3(static_cast<unsigned>(grid), shares),
                       dim3(kMxWaves * 64), static_cast<unsigned>(a.red + kSums), s, a, epi);
    return hipGetLastError();
}

template <typename T, int FMT>
hipError_t launch_small(MxSmallArgs a, const LayerEpilogue<T> &epi, hipStream_t s) {
    // up to eight tiles of rows to a workgroup, and about as many for each
    const int shares = (a.nbt + 7) / 8;
    a.per = (a.nbt + shares - 1) / shares;
    if (a.x) return launch_small_as<T, FMT, 1, true>(a, epi, s);
    if (a.per == 1) return launch_small_as<T, FMT, 1, false>(a, epi, s);
    if (a.per == 2) return launch_small_as<T, FMT, 2, false>(a, epi, s);
    if (a.per <= 4) return launch_small_as<T, FMT, 4, false>(a, epi, s);
    return launch_small_as<T, FMT, 8, false>(a, epi, s);
}

// Tile and splits of the product of B rows of 4-bit codes with M over `steps` steps of 256 columns.
// 256 x 256 tiles where they are at least half as many as compute units (us per call in a graph,
// they / 128 x 128: 2048 x 4096 x 4096 47.0 / 48.1, 1024 x 14336 x 4096 47.9 / 79.2, 4096^3 55.6 /
// 84.0; with 64 tiles, 1024 x 4096 x 4096, 43.0 / 29.0).  Else 128 x 128, whose columns are split
// in two where at most half the compute units have a tile, if there are steps enough (512 x 4096 x
// 14336 38.9 split / 50.1 whole, 512 x 4096 x 4096, 16 steps, 27.6 / 26.1).  Tiles are never fewer
// than 113: smaller products are mx_small_kernel's.
struct MxPlan {
    bool big;
    int splits, steps, steps_per_split;
    int64_t part_ld;
};
constexpr int64_t kMxHalf = 128;    // half the compute units
constexpr int64_t kMxSplitSteps = 24;
MxPlan mx_plan(int64_t B, int64_t M, int64_t steps) {
    MxPlan p{};
    p.steps = static_cast<int>(steps);
    p.part_ld = (M + 3) / 4 * 4;
    p.big = ((B + 255) / 256) * ((M + 255) / 256) >= kMxHalf;
    const int64_t tiles = ((B + 127) / 128) * ((M + 127) / 128);
    p.splits = !p.big && tiles <= kMxHalf && steps >= kMxSplitSteps ? 2 : 1;
    p.steps_per_split = (p.steps + p.splits - 1) / p.splits;
    return p;
}
// Room for the shares, never less for a larger B.
size_t mx_shares(int64_t B, int64_t M, int64_t steps) {
    if (steps < kMxSplitSteps) return 0;
    const int64_t values = 2 * B * ((M + 3) / 4 * 4), most = 2 * kMxHalf * 128 * 128;
    return static_cast<size_t>(values < most ? values : most) * sizeof(float);
}

template <int TI, int TJ, int WI, int WJ, int NB, typename Epi>
hipError_t launch_mx_tiles(const Operand<CodePair> &A, const uint8_t *as,
                           const Operand<CodePair> &W, const uint8_t *ws, const MxPlan &p,
                           const Epi &epi, hipStream_t s) {
    const uint32_t ni = static_cast<uint32_t>((A.rows + TI - 1) / TI);
    const uint32_t nj = static_cast<uint32_t>((W.rows + TJ - 1) / TJ);
    hipLaunchKernelGGL((mx_gemm_kernel<TI, TJ, WI, WJ, NB, Epi>),
                       dim3(ni * nj, static_cast<unsigned>(p.splits)), dim3(WI * WJ * 64), 0, s, A,
                       as, W, ws, p.steps, p.steps_per_split, epi, ni, nj);
    return hipGetLastError();
}

template <typename T>
hipError_t large_fp4(const MxLinearCall &c, const MxMatrix &x, const MxLayout &lay, char *ws,
                     hipStream_t s) {
    const int64_t groups = groups_of(c.N), steps = (groups + 7) / 8;
    const int64_t xt = (c.B + 127) / 128, wt = (c.M + 127) / 128;
    uint8_t *xs = reinterpret_cast<uint8_t *>(ws + lay.xs);
    uint8_t *wsc = xs + pad(xt, 2) * steps * 1024;
    // (256 x 256 tiles read whole pairs of 128 rows)
    const ScaleArgs sx{x.scale, c.B, groups, static_cast<uint32_t>(steps), xs,
                       static_cast<int64_t>(pad(xt, 2)) * steps * 16};
    const ScaleArgs sw{c.w.scale, c.M, groups, static_cast<uint32_t>(steps), wsc,
                       static_cast<int64_t>(pad(wt, 2)) * steps * 16};
    hipError_t e;
    if (steps > 0) {
        hipLaunchKernelGGL(order_scales_kernel,
                           dim3(static_cast<unsigned>((sx.work + sw.work + 255) / 256)),
                           dim3(256), 0, s, sx, sw);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const Operand<CodePair> A{reinterpret_cast<const CodePair *>(x.codes), x.ld, c.B, groups * 16};
    const Operand<CodePair> W{reinterpret_cast<const CodePair *>(c.w.codes), c.w.ld, c.M,
                              groups * 16};
    const MxPlan p = mx_plan(c.B, c.M, steps);
    const LayerEpilogue<T> epi = mx_epilogue<T>(c);
    if (p.big) return launch_mx_tiles<256, 256, 2, 4, gemm::kRing>(A, xs, W, wsc, p, epi, s);
    if (p.splits == 1) return launch_mx_tiles<128, 128, 2, 2, 4>(A, xs, W, wsc, p, epi, s);
    const PartEpilogue pe{reinterpret_cast<float *>(ws + lay.parts), p.part_ld, c.B, c.M};
    e = launch_mx_tiles<128, 128, 2, 2, 4>(A, xs, W, wsc, p, pe, s);
    if (e != hipSuccess) return e;
    const int64_t quads = c.B * (p.part_ld / 4);
    hipLaunchKernelGGL(split_sum_kernel<LayerEpilogue<T>>,
                       dim3(static_cast<unsigned>((quads + 255) / 256)), dim3(256), 0, s, pe.part,
                       p.splits, c.B, p.part_ld, epi);
    return hipGetLastError();
}

// The layer for rows that mx_small_kernel takes, or not.
template <typename T>
hipError_t linear_rows(const MxLinearCall &c, const MxLayout &lay, bool small, char *ws,
                       hipStream_t s) {
    const bool fp4 = c.xq.format == TCQ_FP4;
    const bool dense = small && small_dense(c);
    MxMatrix x = c.xq;
    uint16_t *xvals = reinterpret_cast<uint16_t *>(ws + lay.xvals);
    // (large batches of 8-bit rows are read as the bf16 numbers that the codes stand for, small
    // ones of either in the order of mx_small_kernel's lanes)
    const bool values = !small && !fp4;
    const int64_t groups = groups_of(c.N), pairs = pairs_of(groups);
    const int nbt = static_cast<int>((c.B + 15) / 16);
    const MxOrder order{reinterpret_cast<uint8_t *>(ws + lay.codes),
                        reinterpret_cast<uint8_t *>(ws + lay.scale), nbt};
    hipError_t e;
    if (c.x && !dense) {
        if (!c.keep) {
            x.codes = reinterpret_cast<uint8_t *>(ws + lay.codes);
            x.ld = lay.ldq;
            x.scale = reinterpret_cast<uint8_t *>(ws + lay.scale);
        }
        const bool codes = c.keep || (!values && !small);
        e = launch_mx_pack(c.x, c.dtype, c.B, c.N, c.ldx, c.xq.format,
                           codes ? const_cast<uint8_t *>(x.codes) : nullptr, x.ld,
                           codes ? const_cast<uint8_t *>(x.scale) : nullptr,
                           values ? xvals : nullptr, lay.ldn, small ? &order : nullptr, s);
        if (e != hipSuccess) return e;
    }
    if (small) {
        if (!c.x && c.N > 0) {
            const int64_t work = pairs * nbt * 128 * (fp4 ? 1 : 2);
            hipLaunchKernelGGL(fp4 ? order_rows_kernel<TCQ_FP4> : order_rows_kernel<TCQ_FP8>,
                               dim3(blocks_for(work)), dim3(256), 0, s, x.codes, x.ld, x.scale,
                               static_cast<int>(c.B), static_cast<int>(groups), order, work);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        MxSmallArgs a{};
        a.w = c.w.codes;
        a.ws = c.w.scale;
        a.ldw = c.w.ld;
        a.M = c.M;
        a.N = static_cast<int>(c.N);
        a.groups = static_cast<int>(groups);
        a.pairs = static_cast<int>(pairs);
        a.tiles = static_cast<int>((c.M + 15) / 16);
        a.x = dense ? c.x : nullptr;
        a.ldx = c.ldx;
        a.xq = order.codes;
        a.xs = reinterpret_cast<const uint16_t *>(order.scale);
        a.B = static_cast<int>(c.B);
        a.nbt = nbt;
        a.ldl = dense ? dense_row(c.xq.format, pairs) : 0;
        const LayerEpilogue<T> epi = mx_epilogue<T>(c);
        return fp4 ? launch_small<T, TCQ_FP4>(a, epi, s) : launch_small<T, TCQ_FP8>(a, epi, s);
    }
    if (fp4) return large_fp4<T>(c, x, lay, ws, s);
    if (!c.x) {
        e = launch_mx_unpack(x, c.B, c.N, TCQ_BF16, xvals, lay.ldn, lay.ldn, s);
        if (e != hipSuccess) return e;
    }
    uint16_t *wvals = reinterpret_cast<uint16_t *>(ws + lay.wvals);
    e = launch_mx_unpack(c.w, c.M, c.N, TCQ_BF16, wvals, lay.ldn, lay.ldn, s);
    if (e != hipSuccess) return e;
    const DenseProduct d{xvals,  wvals,      lay.ldn, lay.ldn, c.B, c.M, lay.ldn,
                         c.dtype, c.bias, c.residual, c.ldr,   c.y, c.ldy};
    return launch_dense_product(d, ws + lay.parts, s);
}

// Bytes between the rows of codes up to which a tile's offsets fit CodeLoader's 32 bits: 255 rows
// of it, and a row's last piece, lie below the largest extent of a buffer.  Codes further apart are
// multiplied by mx_small_kernel, whose offsets have 64 bits, in pieces of so many rows that its
// grid holds their shares.
constexpr int64_t kMostPitch = 1 << 24;
static_assert(255 * kMostPitch + 128 < 0xFFFFFF00ll, "offsets of a tile");
constexpr int64_t kFarRows = 1 << 19;

template <typename T>
hipError_t linear(const MxLinearCall &c, char *ws, hipStream_t s) {
    const MxLayout lay = mx_linear_layout(c.xq.format, c.B, c.M, c.N);
    const bool small = mx_small(c.xq.format, c.B, c.M);
    const bool far = c.w.ld > kMostPitch || ((!c.x || c.keep) && c.xq.ld > kMostPitch);
    if (small || c.xq.format != TCQ_FP4 || !far || c.N == 0)
        return linear_rows<T>(c, lay, small, ws, s);
    const int64_t groups = groups_of(c.N);
    for (int64_t b = 0; b < c.B; b += kFarRows) {
        MxLinearCall p = c;
        p.B = c.B - b < kFarRows ? c.B - b : kFarRows;
        if (c.x) p.x = static_cast<const T *>(c.x) + b * c.ldx;
        if (!c.x || c.keep) {
            p.xq.codes += b * c.xq.ld;
            p.xq.scale += b * groups;
        }
        if (c.residual) p.residual = static_cast<const T *>(c.residual) + b * c.ldr;
        p.y = static_cast<T *>(c.y) + b * c.ldy;
        const hipError_t e = linear_rows<T>(p, lay, true, ws, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- gradients

// fp16 holds the values times the power of two that brings the largest finite scale's largest
// code next to the type's own largest number (1.75 2^15), so that none overflows and only those
// 2^-36 of it are rounded; the sums are multiplied by its inverse.  tops[block] = the largest scale
// byte but 255 of the block's share; whoever unpacks takes the largest of them.  (4096^3: 5.1 us
// with 16 workgroups to a matrix, 152 with one.)
struct TopArgs {
    const uint8_t *scale;
    int64_t n;
    int *tops;
};
__global__ __launch_bounds__(1024) void scale_tops_kernel(TopArgs w, TopArgs x) {
    const TopArgs &a = blockIdx.y == 0 ? w : x;
    __shared__ int red[16];
    int top = 0;
    const auto take = [&](uint32_t e) {
        if (e != 255 && static_cast<int>(e) > top) top = static_cast<int>(e);
    };
    struct __attribute__((packed)) Sixteen { uint32_t v[4]; };
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x) * 16; i < a.n;
         i += kMxTops * 1024 * 16) {
        if (i + 16 <= a.n) {
            const Sixteen q = *reinterpret_cast<const Sixteen *>(a.scale + i);
#pragma unroll
            for (int k = 0; k < 16; ++k) take(q.v[k / 4] >> (8 * (k % 4)) & 255u);
        } else {
            for (int64_t k = i; k < a.n; ++k) take(a.scale[k]);
        }
    }
    for (int d = 32; d; d >>= 1) {
        const int o = __shfl_xor(top, d);
        top = top > o ? top : o;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int v = 1; v < 16; ++v) top = top > red[v] ? top : red[v];
        a.tops[blockIdx.x] = top;
    }
}

// The bias' sums from their slabs, W's values and x's, which know nothing of one another, side by
// side in one launch (509 x 2048 x 2048 bf16: three launches 11.5 us, one 5.6).
struct ReadyArgs {
    const float *part;
    int64_t slabs, M;
    float *sum;
    uint32_t sums, w_blocks;    // workgroups of the first two; the others take x
    MxUnpackArgs w, x;
    void *w_out, *x_out;
};
template <typename T, int FMT, bool SMALL>
__global__ __launch_bounds__(256) void grad_ready_kernel(ReadyArgs a) {
    const uint32_t block = blockIdx.x;
    if (block < a.sums)
        slab_sum(a.part, a.slabs, a.M, a.sum, block);
    else if (block - a.sums < a.w_blocks)
        mx_unpack<T, TCQ_FP4, SMALL>(a.w, static_cast<T *>(a.w_out), block - a.sums, a.w_blocks);
    else
        mx_unpack<T, FMT, SMALL>(a.x, static_cast<T *>(a.x_out), block - a.sums - a.w_blocks,
                                 gridDim.x - a.sums - a.w_blocks);
}

template <typename T>
hipError_t grad_ready(const MxGrad &c, ReadyArgs a, int64_t ldn, bool read_w, bool read_x,
                      const int *tops, int *down, hipStream_t s) {
    a.sums = c.dbias && c.M > 0 ? static_cast<uint32_t>((c.M + 63) / 64) : 0;
    uint32_t x_blocks = 0;
    if (read_w) {
        a.w = mx_unpack_args<T>(c.w, c.M, c.N, ldn, ldn);
        a.w_blocks = blocks_for(a.w.ix.total);
        if (__is_same(T, _Float16)) a.w.shift = MxShift{tops, down};
    }
    if (read_x) {
        a.x = mx_unpack_args<T>(c.x, c.B, c.N, ldn, ldn);
        x_blocks = blocks_for(a.x.ix.total);
        if (__is_same(T, _Float16)) a.x.shift = MxShift{tops + kMxTops, down + 1};
    }
    const uint32_t blocks = a.sums + a.w_blocks + x_blocks;
    if (blocks == 0) return hipSuccess;
    const bool small = a.w.ix.total < (int64_t{1} << 32) && a.x.ix.total < (int64_t{1} << 32);
    const auto kern = c.x.format == TCQ_FP4
                          ? (small ? grad_ready_kernel<T, TCQ_FP4, true>
                                   : grad_ready_kernel<T, TCQ_FP4, false>)
                          : (small ? grad_ready_kernel<T, TCQ_FP8, true>
                                   : grad_ready_kernel<T, TCQ_FP8, false>);
    hipLaunchKernelGGL(kern, dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

struct MxGradLayout {
    size_t shifts, w, x, dense, bytes;
    int64_t ldn;
};
MxGradLayout mx_grad_layout(size_t size, int64_t B, int64_t M, int64_t N, bool dx, bool dw,
                            bool dbias) {
    MxGradLayout l{};
    l.ldn = static_cast<int64_t>(pad(N, 8));
    size_t off = 0;
    l.shifts = off;
    if ((dx || dw) && size == 2) off += 256;
    l.w = off;
    if (dx) off += align_up(static_cast<size_t>(M) * l.ldn * size, 256);
    l.x = off;
    if (dw) off += align_up(static_cast<size_t>(B) * l.ldn * size, 256);
    l.dense = off;
    l.bytes = off + dense_grad_layout(size, B, M, N, dx, dw, dbias).bytes;
    return l;
}

}  // namespace

// Codes and scales of x, the ordered scales (4-bit rows) or the bf16 matrices (8-bit), and
// shares: nothing is smaller for a larger B.
MxLayout mx_linear_layout(int format, int64_t B, int64_t M, int64_t N) {
    MxLayout l{};
    const int64_t groups = groups_of(N), steps = (groups + 7) / 8;
    const bool fp4 = format == TCQ_FP4, large = !mx_small(format, B, M);
    l.ldq = groups * (fp4 ? 16 : 32);
    l.ldn = groups * mx::kGroup;
    size_t off = 0;
    // (in the lanes' order whole tiles of 16 rows and whole pairs)
    const int64_t rows = (B + 15) / 16 * 16, whole = pairs_of(groups) * 8;
    l.codes = off;
    off += align_up(static_cast<size_t>(rows) * whole * (fp4 ? 16 : 32), 256);
    l.scale = off;
    off += align_up(static_cast<size_t>(rows) * whole, 256);
    l.xs = l.wvals = l.xvals = l.parts = off;
    if (large && fp4) {
        const size_t tiles = pad((B + 127) / 128, 2) + pad((M + 127) / 128, 2);
        off += tiles * steps * 1024;
        l.parts = off;
        off += align_up(mx_shares(B, M, steps), 256);
    } else if (large) {
        off += align_up(static_cast<size_t>(M) * l.ldn * 2, 256);
        l.xvals = off;
        off += align_up(static_cast<size_t>(B) * l.ldn * 2, 256);
        l.parts = off;
        off += align_up(gemm_shares(2, B, M, l.ldn, 1), 256);
    }
    l.bytes = off;
    return l;
}

hipError_t launch_mx_linear(const MxLinearCall &c, char *ws, hipStream_t s) {
    switch (c.dtype) {
        case TCQ_F32: return linear<float>(c, ws, s);
        case TCQ_F16: return linear<_Float16>(c, ws, s);
        default: return linear<__bf16>(c, ws, s);
    }
}

size_t mx_grad_bytes(int dtype, int64_t B, int64_t M, int64_t N, bool dx, bool dw, bool dbias) {
    return mx_grad_layout(dtype == TCQ_F32 ? 4 : 2, B, M, N, dx, dw, dbias).bytes;
}

hipError_t launch_mx_grad(const MxGrad &c, char *ws, hipStream_t s) {
    const MxGradLayout lay = mx_grad_layout(c.dtype == TCQ_F32 ? 4 : 2, c.B, c.M, c.N, c.dx, c.dw,
                                            c.dbias);
    int *tops = reinterpret_cast<int *>(ws + lay.shifts);   // W's, x's, and the two exponents
    int *down = tops + 2 * kMxTops;
    const bool shifted = c.dtype == TCQ_F16;
    const bool dx = c.dx && c.B > 0 && c.N > 0, dw = c.dw && c.M > 0 && c.N > 0;
    const bool read_w = dx && c.M > 0, read_x = dw && c.B > 0;
    hipError_t e;
    if (shifted && (read_w || read_x)) {
        const int64_t groups = groups_of(c.N);
        const TopArgs w{c.w.scale, c.M * groups, tops};
        const TopArgs x{c.x.scale, c.B * groups, tops + kMxTops};
        hipLaunchKernelGGL(scale_tops_kernel, dim3(kMxTops, read_w && read_x ? 2 : 1), dim3(1024),
                           0, s, read_w ? w : x, x);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const DenseGrad d{c.dtype, c.dy,
                      c.B,     c.lddy,
                      c.M,     c.N,
                      ws + lay.w, ws + lay.x,
                      shifted && read_w ? down : nullptr,
                      shifted && read_x ? down + 1 : nullptr,
                      dx ? c.dx : nullptr, c.lddx,
                      dw ? c.dw : nullptr, c.lddw,
                      c.dbias};
    char *dense = ws + lay.dense;
    e = launch_dense_slabs(d, dense, s);
    if (e != hipSuccess) return e;
    const DenseGradLayout dl = dense_grad_layout(c.dtype == TCQ_F32 ? 4 : 2, c.B, c.M, c.N, d.dx,
                                                 d.dw, d.dbias);
    ReadyArgs a{};
    a.part = reinterpret_cast<const float *>(dense + dl.part);
    a.slabs = dl.slabs;
    a.M = c.M;
    a.sum = c.dbias;
    a.w_out = ws + lay.w;
    a.x_out = ws + lay.x;
    switch (c.dtype) {
        case TCQ_F32: e = grad_ready<float>(c, a, lay.ldn, read_w, read_x, tops, down, s); break;
        case TCQ_F16: e = grad_ready<_Float16>(c, a, lay.ldn, read_w, read_x, tops, down, s); break;
        default: e = grad_ready<__bf16>(c, a, lay.ldn, read_w, read_x, tops, down, s); break;
    }
    if (e != hipSuccess) return e;
    return launch_dense_grad(d, dense, s);
}

}  // namespace tcq
