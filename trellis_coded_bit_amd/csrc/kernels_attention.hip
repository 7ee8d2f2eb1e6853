// Attention of new tokens over the paged, quantised cache (tcq_cache_attention):
//     o[i] = sum_j p[i][j] v[j] / sum_j p[i][j],   p[i][j] = exp(scale q[i] . k[j] - m[i])
// over the keys j that row i sees, in one pass over the cache with the running maximum m and sum
// of a softmax.  The group query heads that share a head of keys are rows of the same product, so
// a key is read once for all of them.
//
// Every code times its scale is a bf16 number, so keys and values are multiplied as bf16 with
// exact products and fp32 sums.  q and p are held in terms of bf16 whose sum they are: one for
// bf16 queries (q is exact; p is rounded to 8 bits, half a step of the output's own type, while
// its sum is taken unrounded), two for fp16 (q exact, p to 2^-15) and three for fp32 (both exact).
//
// Scores are computed transposed, S^T = K Q^T: a lane holds four keys of one query row, the same
// row in every instruction, so a row's maximum and sum are the lane's own but for three other
// lanes, and p is in place as the second operand of O^T = V^T P^T.  That product's order of
// keys is the one the lanes hold them in, and V is read across through LDS in the same order.
//
// Work is cut into items (sequence, head, tile of query rows, run of keys) by every workgroup
// from the lengths on the device, so that the host need not know them: runs are as long as lets
// about kTarget items remain.  A tile with one run writes its outputs, others their share, and
// a second kernel joins shares in the order of the runs.
#include <hip/hip_runtime.h>

#include "cache_device.h"
#include "gemm_device.h"
#include "linear_device.h"
#include "mx_device.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

using gemm::f32x4;
using gemm::s16x4;
using gemm::s16x8;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct AttArgs {
    CacheShape c;
    CacheBatch b;
    CacheRows q, o;
    int group;
    int64_t rows;
    float factor, factor_low;   // scale log2(e), and what it lacks
    float *part;                // shares: [slot][rows of a tile][dim], then maxima and sums
    int64_t slots;
    int both;                   // tiles of 16 rows serve sequences of up to 16 rows only, larger
                                // tiles the others (0: this kernel serves every sequence)
};

// ---------------------------------------------------------------- items

// What a launch of tiles of BQ rows and units of UNIT keys does with a sequence.
struct Sequence {
    int64_t tiles, units, chunks;
};
constexpr int kUnit = 128;      // keys: runs are whole units
constexpr int kSmallRows = 16;
constexpr int64_t kTargetSmall = 1024, kTargetLarge = 512;
template <int BQ>
constexpr int64_t target() {
    return BQ == kSmallRows ? kTargetSmall : kTargetLarge;
}

template <int BQ>
__device__ __forceinline__ Sequence sequence(const AttArgs &a, int64_t s) {
    Sequence r{0, 0, 1};
    if (s >= a.b.seqs) return r;
    const cache::Span sp = cache::span_of(a.b, s, a.rows);
    const int64_t n = sp.end - sp.begin;
    if (n <= 0) return r;
    const bool small = n * a.group <= kSmallRows;
    if (a.both && small != (BQ == kSmallRows)) return r;
    r.tiles = (n * a.group + BQ - 1) / BQ;
    int64_t keys = sp.first + n;  // the last row sees the keys before this
    const int64_t most = a.b.width << a.c.page_log2;
    keys = keys < 0 ? 0 : (keys < most ? keys : most);
    r.units = (keys + kUnit - 1) / kUnit;
    return r;
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ int64_t wave_prefix(int64_t v, int lane) {
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Units per run: the fewest with at most about the target number of runs in all.
template <int BQ>
__device__ __forceinline__ int64_t run_units(const AttArgs &a, int lane) {
    int64_t total = 0;
    for (int64_t s = 0; s < a.b.seqs; s += 64) {
        const Sequence q = sequence<BQ>(a, s + lane);
        total += q.tiles * q.units;
    }
    total = wave_sum(total) * a.c.heads;
    const int64_t per = (total + target<BQ>() - 1) / target<BQ>();
    return per > 1 ? per : 1;
}

struct Item {
    int64_t seq, tile, chunk, chunks;
    int head;
    int64_t slot;       // of its share (chunks > 1)
    int64_t begin, end; // keys of the run
};

// Item `index`, or false past the last.  Heads vary fastest, so that those of one sequence go
// to different XCDs and a head's tiles to the same one, then tiles, later ones (more keys) first.
template <int BQ>
__device__ __forceinline__ bool item_of(const AttArgs &a, int64_t index, int lane, Item &it) {
    const int64_t per = run_units<BQ>(a, lane);
    int64_t slots = 0;
    for (int64_t s = 0; s < a.b.seqs; s += 64) {
        Sequence q = sequence<BQ>(a, s + lane);
        q.chunks = q.units > per ? (q.units + per - 1) / per : 1;
        const int64_t n = q.tiles * q.chunks * a.c.heads, shared = q.chunks > 1 ? n : 0;
        const int64_t to = wave_prefix(n, lane), all = __shfl(to, 63);
        if (index < all) {
            const int64_t stop = wave_prefix(shared, lane);
            const int at = __popcll(__ballot(to <= index));  // lanes before the item's
            const int64_t left = index - (__shfl(to, at) - __shfl(n, at));
            const int64_t tiles = __shfl(q.tiles, at);
            it.seq = s + at;
            it.chunks = __shfl(q.chunks, at);
            it.slot = slots + __shfl(stop, at) - __shfl(shared, at) + left;
            it.head = static_cast<int>(left % a.c.heads);
            const int64_t rest = left / a.c.heads;
            it.tile = tiles - 1 - rest % tiles;
            it.chunk = rest / tiles;
            it.begin = it.chunk * per * kUnit;
            it.end = it.chunk + 1 < it.chunks ? it.begin + per * kUnit : INT64_MAX;
            return true;
        }
        index -= all;
        slots += wave_sum(shared);
    }
    return false;
}

// ---------------------------------------------------------------- numbers

// a and b in TERMS bf16 terms, a in the low half of each word.  All but the last cut off bits
// (so a number next to the largest stays finite); one or two terms round the last to nearest,
// three hold every bit.
template <int TERMS>
__device__ __forceinline__ void terms_of(float a, float b, uint32_t (&w)[TERMS]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int t = 0; t + 1 < TERMS; ++t) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        w[t] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);  // the upper halves
        a -= __uint_as_float(ua & 0xFFFF0000u);             // exact
        b -= __uint_as_float(ub & 0xFFFF0000u);
    }
    if constexpr (TERMS == 3)
        w[2] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    else
        w[TERMS - 1] =
            __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

template <typename T>
constexpr int terms() {
    return sizeof(T) == 4 ? 3 : (__is_same(T, _Float16) ? 2 : 1);
}

// The largest (sum) over the four lanes that hold a query row's keys: lanes l, l ^ 16, l ^ 32.
__device__ __forceinline__ float row_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16));
    return __builtin_fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// The running softmax of one query row per lane.
struct Softmax {
    float top;    // the largest score so far times factor
    float sum;    // of this lane's keys
    __device__ __forceinline__ void init() {
        top = -__builtin_inff();
        sum = 0.0f;
    }
    // What p is taken relative to: 2^-top, and 1 before the first key.
    static __device__ __forceinline__ float safe(float t) {
        return t == -__builtin_inff() ? 0.0f : t;
    }
};

// p = 2^(s factor - top); fp32 takes what the factor lacks along.
template <int TERMS>
__device__ __forceinline__ float weight(float s, float factor, float low, float top) {
    float e = __builtin_fmaf(s, factor, -top);
    if constexpr (TERMS == 3) {
        // (masked keys: -inf, whose product with low would be NaN)
        e = __builtin_fmaf(__builtin_fmaxf(s, -0x1p127f), low, e);
    }
    return __builtin_amdgcn_exp2f(e);
}

// Reads A = X^T (16 columns from unit `unit` of 32 bytes, 32 rows r0 ..) from a tile of X in LDS,
// rows of W bytes, whose units are permuted by the row: row 4 g + i in place i and row 16 + 4 g
// + i in place 4 + i of lane group g.
template <int W>
__device__ __forceinline__ s16x8 read_across(const char *lds, int r0, int unit, int lane) {
    typedef __attribute__((address_space(3))) s16x4 *P;
    constexpr int kMask = W / 32 < 8 ? W / 32 - 1 : 7;
    const int l16 = lane & 15, g = lane >> 4;
    s16x8 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * h + 4 * g + (l16 >> 2);
        const char *p = lds + (r0 + r) * W + (unit ^ (r & kMask)) * 32 + (l16 & 3) * 8;
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
#pragma unroll
        for (int v = 0; v < 4; ++v) out[h * 4 + v] = t[v];
    }
    return out;
}
template <int W>
__device__ __forceinline__ char *unit_at(char *lds, int row, int unit) {
    constexpr int kMask = W / 32 < 8 ? W / 32 - 1 : 7;
    return lds + row * W + (unit ^ (row & kMask)) * 32;
}

// 16 bytes of codes (16 of fp8, 32 of fp4) to bf16 words.
template <int FMT>
__device__ __forceinline__ void decode16(const u32x4 &q, float s, uint32_t *w) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        mx::decode_word_bf16<FMT>(q[j], s, w + (FMT == TCQ_FP4 ? 4 : 2) * j);
}

// ---------------------------------------------------------------- outputs

// Shares of a tile: BQ x D sums, then BQ maxima and BQ sums of weights.
template <int BQ, int D>
constexpr int64_t slot_floats() {
    return BQ * (D + 2);
}

// Four consecutive outputs d .. d + 3 of query row r of the tile: written as they are (a single
// run) or as a share.
template <typename T, int BQ, int D>
struct Output {
    const AttArgs &a;
    const Item &it;
    cache::Span sp;
    float *slot;
    __device__ __forceinline__ Output(const AttArgs &a_, const Item &it_, const cache::Span &sp_)
        : a(a_), it(it_), sp(sp_) {
        slot = it.chunks > 1 ? a.part + it.slot * slot_floats<BQ, D>() : nullptr;
    }
    __device__ __forceinline__ bool room() const { return it.chunks == 1 || it.slot < a.slots; }
    __device__ __forceinline__ void put(int r, int d, f32x4 o, float top, float sum) const {
        if (slot) {
            *reinterpret_cast<f32x4 *>(slot + r * D + d) = o;
            if (d == 0) {
                slot[BQ * D + r] = top;
                slot[BQ * D + BQ + r] = sum;
            }
            return;
        }
        store(a, it.seq, it.head, it.tile * BQ + r, sp, d, o, sum);
    }
    // (a row that saw no key: zeros)
    static __device__ __forceinline__ void store(const AttArgs &a, int64_t, int head, int64_t r,
                                                 const cache::Span &sp, int d, f32x4 o,
                                                 float sum) {
        const int64_t i = r / a.group, row = sp.begin + i;
        if (row >= sp.end) return;
        const int64_t h = static_cast<int64_t>(head) * a.group + (r - i * a.group);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        Packed<T, 4> p;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            p.v[v] = static_cast<T>(sum == 0.0f ? 0.0f : o[v] * inv);
        T *out = static_cast<T *>(const_cast<void *>(a.o.p)) + row * a.o.row + h * a.o.head + d;
        *reinterpret_cast<Packed<T, 4> *>(out) = p;
    }
};

// The fragments of query row `r` (this lane's) in terms: place 8 f + v of lane group g holds d =
// at(f) + v.
template <typename T, int D, int TERMS, typename At>
__device__ __forceinline__ void load_query(const AttArgs &a, const Item &it, const cache::Span &sp,
                                           int64_t r, const At &at, s16x8 (&q)[TERMS][D / 32]) {
    const int64_t i = r / a.group, row = sp.begin + i;
    const int64_t h = static_cast<int64_t>(it.head) * a.group + (r - i * a.group);
    const bool in = row < sp.end;
    const T *x = static_cast<const T *>(a.q.p) + row * a.q.row + h * a.q.head;
#pragma unroll
    for (int f = 0; f < D / 32; ++f) {
        float v[8];
        if (in) {
            const Packed<T> p = *reinterpret_cast<const Packed<T> *>(x + at(f));
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(p.v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        u32x4 w[TERMS];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t t[TERMS];
            terms_of<TERMS>(v[2 * k], v[2 * k + 1], t);
#pragma unroll
            for (int n = 0; n < TERMS; ++n) w[n][k] = t[n];
        }
#pragma unroll
        for (int n = 0; n < TERMS; ++n) q[n][f] = __builtin_bit_cast(s16x8, w[n]);
    }
}

// One 16 x 16 product over 32 keys or dims, smallest term first.
template <int TERMS>
__device__ __forceinline__ f32x4 mma_terms(const s16x8 &x, const s16x8 (&y)[TERMS], f32x4 c) {
#pragma unroll
    for (int n = TERMS - 1; n >= 0; --n) c = gemm::Traits<__bf16>::mma(x, y[n], c);
    return c;
}

// ---------------------------------------------------------------- few query rows

// 16 query rows, four waves that take every fourth tile of 32 keys of the run, each with its own
// softmax; joined in LDS.  Keys go from memory straight into the first operand of S^T (a lane
// reads a run of D / 4 dims of its key), values through the wave's own piece of LDS.
template <typename T, int D, int FMT>
__global__ __launch_bounds__(256) void attend_few_kernel(AttArgs a) {
    constexpr int TERMS = terms<T>();
    constexpr int BQ = kSmallRows;
    constexpr int kRow = mx::bytes<FMT>(D);    // bytes of a cache row
    constexpr int kRun = kRow / 4;             // of it, one lane's
    constexpr int kLanes = kRow / 16;          // lanes to a row of values
    constexpr int kVLoads = 32 * kLanes / 64;
    constexpr int kGroups = D / 32;
    constexpr int kTiles = D / 16;             // tiles of 16 dims
    __shared__ __align__(16) char lds[4 * 32 * D * 2];
    __shared__ float tops[4][16], sums[4][16];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Item it;
    if (!item_of<BQ>(a, blockIdx.x, lane, it)) return;
    const cache::Span sp = cache::span_of(a.b, it.seq, a.rows);
    const Output<T, BQ, D> out(a, it, sp);
    if (!out.room()) return;
    const int64_t n_rows = (sp.end - sp.begin) * a.group;
    const int64_t r0 = it.tile * BQ;
    const int64_t last = r0 + BQ < n_rows ? r0 + BQ - 1 : n_rows - 1;
    // keys that some row of the tile sees, and those that all do
    const int64_t capacity = a.b.width << a.c.page_log2;
    int64_t end = sp.first + last / a.group + 1;
    end = end < capacity ? end : capacity;
    end = end < it.end ? end : it.end;
    const int64_t seen_by_all = sp.first + r0 / a.group + 1;
    const int64_t mine = sp.first + (r0 + l16) / a.group;  // the last key that this lane's row sees

    s16x8 q[TERMS][kGroups];
    load_query<T, D, TERMS>(a, it, sp, r0 + l16, [&](int f) { return g * (D / 4) + 8 * f; }, q);

    char *vt = lds + wave * (32 * D * 2);
    // the cache row of the tile's key t (0 .. 31) is held by lane t; -1: not there
    auto rows_at = [&](int64_t base) {
        const int64_t pos = base + (lane & 31);
        if (pos >= end) return int64_t{-1};
        const int64_t page = cache::page_of(a.b, a.c, it.seq, pos);
        return page < 0 ? int64_t{-1} : cache::row_of(a.c, page, it.head, pos);
    };
    struct Codes {
        u32x4 k[2][kRun >= 16 ? kRun / 16 : 1];
        int ke[2][kGroups > 4 ? 2 : 1];
        u32x4 v[kVLoads];
        int ve[kVLoads];
    };
    auto load = [&](int64_t row, Codes &c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = __shfl(row, 16 * h + l16);
            const uint8_t *p = a.c.k_codes + r * kRow + g * kRun;
            const uint8_t *e = a.c.k_scale + r * kGroups + (g * (D / 4)) / 32;
#pragma unroll
            for (int j = 0; j < (kRun >= 16 ? kRun / 16 : 1); ++j) c.k[h][j] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < (kGroups > 4 ? 2 : 1); ++j) c.ke[h][j] = 127;
            if (r >= 0) {
                if constexpr (kRun >= 16) {
#pragma unroll
                    for (int j = 0; j < kRun / 16; ++j)
                        c.k[h][j] = *reinterpret_cast<const u32x4 *>(p + 16 * j);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    c.k[h][0] = u32x4{w.x, w.y, 0, 0};
                }
#pragma unroll
                for (int j = 0; j < (kGroups > 4 ? 2 : 1); ++j) c.ke[h][j] = e[j];
            }
        }
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) {
            const int64_t r = __shfl(row, j * (64 / kLanes) + lane / kLanes);
            const int part = lane % kLanes;
            c.v[j] = u32x4{0, 0, 0, 0};
            c.ve[j] = 127;
            if (r >= 0) {
                c.v[j] = *reinterpret_cast<const u32x4 *>(a.c.v_codes + r * kRow + part * 16);
                c.ve[j] = a.c.v_scale[r * kGroups + part / (kLanes / kGroups)];
            }
        }
    };

    f32x4 acc[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    Softmax sm;
    sm.init();
    int64_t base = it.begin + 32 * wave;
    int64_t row = base < end ? rows_at(base) : -1;
    Codes now;
    if (base < end) load(row, now);
    for (; base < end; base += 128) {
        const uint32_t there = static_cast<uint32_t>(__ballot(row >= 0));
        // scores
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0.f, 0.f, 0.f, 0.f};
            uint32_t w[D / 8];
            if constexpr (FMT == TCQ_FP8) {
#pragma unroll
                for (int j = 0; j < kRun / 16; ++j)
                    decode16<FMT>(now.k[h][j], mx::scale_of(now.ke[h][j / 2]), w + 8 * j);
            } else if constexpr (kRun == 8) {
                mx::decode_word_bf16<FMT>(now.k[h][0][0], mx::scale_of(now.ke[h][0]), w);
                mx::decode_word_bf16<FMT>(now.k[h][0][1], mx::scale_of(now.ke[h][0]), w + 4);
            } else {
#pragma unroll
                for (int j = 0; j < kRun / 16; ++j)
                    decode16<FMT>(now.k[h][j], mx::scale_of(now.ke[h][j]), w + 16 * j);
            }
#pragma unroll
            for (int f = 0; f < kGroups; ++f) {
                const s16x8 x = __builtin_bit_cast(
                    s16x8, (u32x4{w[4 * f], w[4 * f + 1], w[4 * f + 2], w[4 * f + 3]}));
                s16x8 y[TERMS];
#pragma unroll
                for (int n = 0; n < TERMS; ++n) y[n] = q[n][f];
                s[h] = mma_terms<TERMS>(x, y, s[h]);
            }
        }
        // values into LDS; what stands for NaN goes in as zero and is added below
        bool wild = false;
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) {
            const int r = j * (64 / kLanes) + lane / kLanes, part = lane % kLanes;
            wild |= now.ve[j] == 255;
            const float sc = mx::scale_of(now.ve[j]);
            constexpr int kWords = FMT == TCQ_FP4 ? 16 : 8;
            uint32_t w[kWords];
            decode16<FMT>(now.v[j], sc, w);
            if (now.ve[j] == 255) {
#pragma unroll
                for (int k = 0; k < kWords; ++k) w[k] = 0;
            }
#pragma unroll
            for (int u = 0; u < kWords / 8; ++u) {
                u32x4 *p = reinterpret_cast<u32x4 *>(
                    unit_at<D * 2>(vt, r, part * (kWords / 8) + u));
                p[0] = u32x4{w[8 * u], w[8 * u + 1], w[8 * u + 2], w[8 * u + 3]};
                p[1] = u32x4{w[8 * u + 4], w[8 * u + 5], w[8 * u + 6], w[8 * u + 7]};
            }
        }
        int ve[kVLoads];
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) ve[j] = now.ve[j];
        // the next tile's codes
        const int64_t next = base + 128;
        const int64_t next_row = next < end ? rows_at(next) : -1;
        if (next < end) load(next_row, now);
        // mask: keys that are not there, and those past this lane's row
        uint32_t sees = 0xFFu;  // bit 4 h + v: key 16 h + 4 g + v
        if (there != 0xFFFFFFFFu || base + 32 > seen_by_all) {
            sees = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = 16 * (i / 4) + 4 * g + i % 4;
                if ((there >> t & 1) && base + t <= mine) sees |= 1u << i;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(sees >> i & 1)) s[i / 4][i % 4] = -__builtin_inff();
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, s[i / 4][i % 4]);
        top = __builtin_fmaxf(row_max(top) * a.factor, sm.top);
        const float ref = Softmax::safe(top);
        const float alpha = __builtin_amdgcn_exp2f(sm.top - ref);
        sm.top = top;
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = weight<TERMS>(s[i / 4][i % 4], a.factor, a.factor_low, ref);
        float add = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) add += p[i];
        sm.sum = __builtin_fmaf(sm.sum, alpha, add);
        s16x8 pf[TERMS];
        {
            u32x4 w[TERMS];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t t[TERMS];
                terms_of<TERMS>(p[2 * k], p[2 * k + 1], t);
#pragma unroll
                for (int n = 0; n < TERMS; ++n) w[n][k] = t[n];
            }
#pragma unroll
            for (int n = 0; n < TERMS; ++n) pf[n] = __builtin_bit_cast(s16x8, w[n]);
        }
        if (__any(alpha != 1.0f)) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) acc[t] *= alpha;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            acc[t] = mma_terms<TERMS>(read_across<D * 2>(vt, 0, t, lane), pf, acc[t]);
        __builtin_amdgcn_wave_barrier();
        // A value that stands for NaN reaches the rows that see its key, whatever p: counted by
        // the same product over ones.
        if (__builtin_expect(__any(wild), 0)) {
#pragma unroll
            for (int j = 0; j < kVLoads; ++j) {
                const int r = j * (64 / kLanes) + lane / kLanes, part = lane % kLanes;
                constexpr int kUnits = FMT == TCQ_FP4 ? 2 : 1;
                const uint32_t w = ve[j] == 255 ? 0x3F803F80u : 0u;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    u32x4 *d = reinterpret_cast<u32x4 *>(
                        unit_at<D * 2>(vt, r, part * kUnits + u));
                    d[0] = d[1] = u32x4{w, w, w, w};
                }
            }
            u32x4 ones;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                ones[k] = (sees >> (2 * k) & 1 ? 0x3F80u : 0u) |
                          (sees >> (2 * k + 1) & 1 ? 0x3F800000u : 0u);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const f32x4 n = gemm::Traits<__bf16>::mma(read_across<D * 2>(vt, 0, t, lane),
                                                          __builtin_bit_cast(s16x8, ones),
                                                          f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (n[v] != 0.0f) acc[t][v] = __builtin_nanf("");
            }
            __builtin_amdgcn_wave_barrier();
        }
        row = next_row;
    }
    // join the waves
    const float sum = row_sum(sm.sum);
    if (g == 0) {
        tops[wave][l16] = sm.top;
        sums[wave][l16] = sum;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
        reinterpret_cast<f32x4 *>(vt)[t * 64 + lane] = acc[t];
    __syncthreads();
    for (int i = tid; i < 16 * (D / 4); i += 256) {
        const int r = i / (D / 4), d4 = i % (D / 4);
        float top = tops[0][r];
#pragma unroll
        for (int w = 1; w < 4; ++w) top = __builtin_fmaxf(top, tops[w][r]);
        const float ref = Softmax::safe(top);
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        float total = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = __builtin_amdgcn_exp2f(tops[w][r] - ref);
            const f32x4 v = reinterpret_cast<const f32x4 *>(
                lds + w * (32 * D * 2))[(d4 / 4) * 64 + (d4 % 4) * 16 + r];
            total = __builtin_fmaf(sums[w][r], f, total);
            o += v * f;
        }
        out.put(r, d4 * 4, o, top, total);
    }
}

// ---------------------------------------------------------------- many query rows

// 128 query rows, two tiles of 16 to each of four waves, and tiles of 64 keys that the workgroup's
// threads decode into LDS for all waves, with the next tile's codes on their way.
constexpr int kLargeRows = 128;

template <typename T, int D, int FMT>
__global__ __launch_bounds__(256) void attend_many_kernel(AttArgs a) {
    constexpr int TERMS = terms<T>();
    constexpr int NQ = 2, BQ = kLargeRows;
    static_assert(BQ == 4 * NQ * 16, "four waves");
    constexpr int kRow = mx::bytes<FMT>(D);
    constexpr int kLanes = kRow / 16;
    constexpr int kGroups = D / 32;
    constexpr int kTiles = D / 16;
    constexpr int kPieces = 64 * kLanes;                       // of 16 bytes, of a tile
    constexpr int kLoads = (kPieces + 255) / 256;
    constexpr int kWords = FMT == TCQ_FP4 ? 16 : 8;            // of bf16 pairs to a piece
    __shared__ __align__(16) char kt[64 * D * 2];
    __shared__ __align__(16) char vt[64 * D * 2];
    __shared__ unsigned long long absent_of[2];
    __shared__ int wild_of[2];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Item it;
    if (!item_of<BQ>(a, blockIdx.x, lane, it)) return;
    const cache::Span sp = cache::span_of(a.b, it.seq, a.rows);
    const Output<T, BQ, D> out(a, it, sp);
    if (!out.room()) return;
    const int64_t n_rows = (sp.end - sp.begin) * a.group;
    const int64_t r0 = it.tile * BQ + wave * (NQ * 16);
    const int64_t tile_last = it.tile * BQ + BQ < n_rows ? it.tile * BQ + BQ - 1 : n_rows - 1;
    const int64_t capacity = a.b.width << a.c.page_log2;
    int64_t end = sp.first + tile_last / a.group + 1;
    end = end < capacity ? end : capacity;
    end = end < it.end ? end : it.end;
    const int64_t seen_by_all = sp.first + r0 / a.group + 1;
    int64_t mine[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) mine[n] = sp.first + (r0 + 16 * n + l16) / a.group;
    s16x8 q[NQ][TERMS][kGroups];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
        load_query<T, D, TERMS>(a, it, sp, r0 + 16 * n + l16,
                                [&](int f) { return 32 * f + 8 * g; }, q[n]);

    // pieces of this thread: key p / kLanes, bytes 16 (p % kLanes) of its row
    struct Codes {
        int64_t row[kLoads];
        u32x4 k[kLoads], v[kLoads];
        int ke[kLoads], ve[kLoads];
    } now;
    auto find = [&](int64_t base) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int p = j * 256 + tid;
            const int64_t pos = base + p / kLanes;
            now.row[j] = -1;
            if (p < kPieces && pos < end) {
                const int64_t page = cache::page_of(a.b, a.c, it.seq, pos);
                if (page >= 0) now.row[j] = cache::row_of(a.c, page, it.head, pos);
            }
        }
    };
    auto load = [&] {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int part = (j * 256 + tid) % kLanes;
            now.k[j] = now.v[j] = u32x4{0, 0, 0, 0};
            now.ke[j] = now.ve[j] = 127;
            if (now.row[j] >= 0) {
                const int64_t at = now.row[j] * kRow + part * 16;
                const int64_t e = now.row[j] * kGroups + part / (kLanes / kGroups);
                now.k[j] = *reinterpret_cast<const u32x4 *>(a.c.k_codes + at);
                now.v[j] = *reinterpret_cast<const u32x4 *>(a.c.v_codes + at);
                now.ke[j] = a.c.k_scale[e];
                now.ve[j] = a.c.v_scale[e];
            }
        }
    };
    // K: 16-byte chunks of a row permuted by the row
    auto chunk_at = [&](int row, int chunk) {
        return reinterpret_cast<u32x4 *>(kt + row * (D * 2) + (chunk ^ (row & 7)) * 16);
    };
    f32x4 acc[NQ][kTiles];
    Softmax sm[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        sm[n].init();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    int64_t base = it.begin;
    if (base < end) {
        find(base);
        load();
    }
    if (tid < 2) absent_of[tid] = 0, wild_of[tid] = 0;
    __syncthreads();
    int turn = 0;
    for (; base < end; base += 64, turn ^= 1) {
        // codes into LDS
        bool wild = false;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int p = j * 256 + tid;
            const int r = p / kLanes, part = p % kLanes;
            if (p < kPieces) {
                if (now.row[j] < 0) atomicOr(&absent_of[turn], 1ull << r);
                uint32_t w[kWords];
                decode16<FMT>(now.k[j], mx::scale_of(now.ke[j]), w);
#pragma unroll
                for (int u = 0; u < kWords / 4; ++u)
                    *chunk_at(r, part * (kWords / 4) + u) =
                        u32x4{w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]};
                decode16<FMT>(now.v[j], mx::scale_of(now.ve[j]), w);
                if (now.ve[j] == 255) {
                    wild = true;
#pragma unroll
                    for (int k = 0; k < kWords; ++k) w[k] = 0;
                }
#pragma unroll
                for (int u = 0; u < kWords / 8; ++u) {
                    u32x4 *d = reinterpret_cast<u32x4 *>(
                        unit_at<D * 2>(vt, r, part * (kWords / 8) + u));
                    d[0] = u32x4{w[8 * u], w[8 * u + 1], w[8 * u + 2], w[8 * u + 3]};
                    d[1] = u32x4{w[8 * u + 4], w[8 * u + 5], w[8 * u + 6], w[8 * u + 7]};
                }
            }
        }
        if (__any(wild) && lane == 0) wild_of[turn] = 1;
        int ve[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) ve[j] = now.ve[j];
        __syncthreads();
        const uint64_t there = ~absent_of[turn];
        const bool any_wild = wild_of[turn] != 0;
        const int64_t next = base + 64;
        if (next < end) {
            find(next);
            load();
        }
        // scores of 64 keys
        f32x4 s[NQ][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < kGroups; ++f) {
                const s16x8 x =
                    __builtin_bit_cast(s16x8, *chunk_at(16 * h + l16, 4 * f + g));
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    s16x8 y[TERMS];
#pragma unroll
                    for (int m = 0; m < TERMS; ++m) y[m] = q[n][m][f];
                    s[n][h] = mma_terms<TERMS>(x, y, s[n][h]);
                }
            }
        }
        s16x8 pf[NQ][2][TERMS];
        uint32_t sees[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            sees[n] = 0xFFFFu;  // bit 4 h + v: key 16 h + 4 g + v
            if (there != ~0ull || base + 64 > seen_by_all) {
                sees[n] = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 16 * (i / 4) + 4 * g + i % 4;
                    if ((there >> t & 1) && base + t <= mine[n]) sees[n] |= 1u << i;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!(sees[n] >> i & 1)) s[n][i / 4][i % 4] = -__builtin_inff();
            }
            float top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[n][i / 4][i % 4]);
            top = __builtin_fmaxf(row_max(top) * a.factor, sm[n].top);
            const float ref = Softmax::safe(top);
            const float alpha = __builtin_amdgcn_exp2f(sm[n].top - ref);
            sm[n].top = top;
            float add = 0.0f;
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = weight<TERMS>(s[n][i / 4][i % 4], a.factor, a.factor_low, ref);
                add += p[i];
            }
            sm[n].sum = __builtin_fmaf(sm[n].sum, alpha, add);
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                u32x4 w[TERMS];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t t[TERMS];
                    terms_of<TERMS>(p[8 * k2 + 2 * k], p[8 * k2 + 2 * k + 1], t);
#pragma unroll
                    for (int m = 0; m < TERMS; ++m) w[m][k] = t[m];
                }
#pragma unroll
                for (int m = 0; m < TERMS; ++m) pf[n][k2][m] = __builtin_bit_cast(s16x8, w[m]);
            }
            if (__any(alpha != 1.0f)) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) acc[n][t] *= alpha;
            }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                const s16x8 x = read_across<D * 2>(vt, 32 * k2, t, lane);
#pragma unroll
                for (int n = 0; n < NQ; ++n) acc[n][t] = mma_terms<TERMS>(x, pf[n][k2], acc[n][t]);
            }
        }
        if (tid == 0) absent_of[turn ^ 1] = 0, wild_of[turn ^ 1] = 0;
        __syncthreads();
        // values that stand for NaN, as in attend_few_kernel
        if (__builtin_expect(any_wild, 0)) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int p = j * 256 + tid;
                if (p < kPieces) {
                    const uint32_t w = ve[j] == 255 ? 0x3F803F80u : 0u;
#pragma unroll
                    for (int u = 0; u < kWords / 8; ++u) {
                        u32x4 *d = reinterpret_cast<u32x4 *>(
                            unit_at<D * 2>(vt, p / kLanes, (p % kLanes) * (kWords / 8) + u));
                        d[0] = d[1] = u32x4{w, w, w, w};
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    u32x4 ones;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ones[k] = (sees[n] >> (8 * k2 + 2 * k) & 1 ? 0x3F80u : 0u) |
                                  (sees[n] >> (8 * k2 + 2 * k + 1) & 1 ? 0x3F800000u : 0u);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        const f32x4 c = gemm::Traits<__bf16>::mma(
                            read_across<D * 2>(vt, 32 * k2, t, lane),
                            __builtin_bit_cast(s16x8, ones), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (c[v] != 0.0f) acc[n][t][v] = __builtin_nanf("");
                    }
                }
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const float sum = row_sum(sm[n].sum);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            out.put(wave * (NQ * 16) + 16 * n + l16, 16 * t + 4 * g, acc[n][t], sm[n].top, sum);
    }
}

// ---------------------------------------------------------------- join of shares

// Rows of tiles with several runs: a wave takes a row, its lanes four dims each; the shares are
// added in the order of the runs.
constexpr int kJoinRows = 16;    // rows to a workgroup of four waves
template <typename T, int D, int BQ>
__device__ __forceinline__ void join(const AttArgs &a, int64_t block) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int kParts = BQ / kJoinRows;
    // (tile of rows with several runs) number `block / kParts`
    const int64_t per = run_units<BQ>(a, lane);
    int64_t index = block / kParts, slots = 0;
    for (int64_t s = 0; s < a.b.seqs; s += 64) {
        Sequence q = sequence<BQ>(a, s + lane);
        q.chunks = q.units > per ? (q.units + per - 1) / per : 1;
        const int64_t pairs = q.chunks > 1 ? q.tiles * a.c.heads : 0, n = pairs * q.chunks;
        const int64_t to = wave_prefix(pairs, lane), all = __shfl(to, 63);
        if (index >= all) {
            index -= all;
            slots += wave_sum(n);
            continue;
        }
        const int64_t stop = wave_prefix(n, lane);
        const int at = __popcll(__ballot(to <= index));
        const int64_t left = index - (__shfl(to, at) - __shfl(pairs, at));
        const int64_t tiles = __shfl(q.tiles, at), chunks = __shfl(q.chunks, at);
        const int64_t heads = a.c.heads;
        // slots of the pair: first + chunk (tiles x heads)
        const int64_t first = slots + __shfl(stop, at) - __shfl(n, at) + left;
        const int head = static_cast<int>(left % heads);
        const int64_t tile = tiles - 1 - left / heads;
        const int64_t stride = tiles * heads;
        if (first + (chunks - 1) * stride >= a.slots) return;
        const cache::Span sp = cache::span_of(a.b, s + at, a.rows);
        for (int i = wave; i < kJoinRows; i += 4) {
            const int r = static_cast<int>(block % kParts) * kJoinRows + i;
            if (tile * BQ + r >= (sp.end - sp.begin) * a.group) break;
            const float *slot = a.part + first * slot_floats<BQ, D>();
            const int64_t step = stride * slot_floats<BQ, D>();
            float top = -__builtin_inff();
            for (int64_t c = lane; c < chunks; c += 64)
                top = __builtin_fmaxf(top, slot[c * step + BQ * D + r]);
            for (int d = 32; d; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
            const float ref = Softmax::safe(top);
            const int d = lane * 4;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            float total = 0.0f;
#pragma unroll 4
            for (int64_t c = 0; c < chunks; ++c) {
                const float *p = slot + c * step;
                const float f = __builtin_amdgcn_exp2f(p[BQ * D + r] - ref);
                total = __builtin_fmaf(p[BQ * D + BQ + r], f, total);
                if (d < D) o += *reinterpret_cast<const f32x4 *>(p + r * D + d) * f;
            }
            if (d < D)
                Output<T, BQ, D>::store(a, s + at, head, tile * BQ + r, sp, d, o, total);
        }
        return;
    }
}
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(AttArgs few, AttArgs many, uint32_t blocks_few) {
    if (blockIdx.x < blocks_few)
        join<T, D, kSmallRows>(few, blockIdx.x);
    else
        join<T, D, kLargeRows>(many, blockIdx.x - blocks_few);
}

// ---------------------------------------------------------------- host side

// Sequences of few rows each (on average up to 16) are all given to the kernel of 16 rows, which
// then reads a sequence's keys at most twice as often as rows of 16 need on average; in other
// batches those of at most 16 rows are.
bool few_only(int64_t rows, int group, int64_t seqs) {
    return rows * group <= kSmallRows * seqs;
}

// Shares: a sequence has several runs only where they are whole runs of about total / target
// units, so there are at most twice the target.
constexpr int64_t kSlotsFew = 2 * kTargetSmall, kSlotsMany = 2 * kTargetLarge;

int64_t slot_bytes(int bq, int dim) { return int64_t{bq} * (dim + 2) * 4; }

template <typename T, int D, int FMT>
hipError_t attend(const AttArgs &base, char *ws, hipStream_t s) {
    AttArgs few = base, many = base;
    const bool only = few_only(base.rows, base.group, base.b.seqs);
    const int64_t heads = base.c.heads;
    few.both = many.both = !only;
    few.part = reinterpret_cast<float *>(ws);
    few.slots = kSlotsFew;
    many.part = reinterpret_cast<float *>(ws + kSlotsFew * slot_bytes(kSmallRows, D));
    many.slots = kSlotsMany;
    // tiles of all sequences: whole ones of the rows, and a part of one for each
    const int64_t qrows = base.rows * base.group;
    const int64_t few_tiles = only ? qrows / kSmallRows + base.b.seqs : base.b.seqs;
    const int64_t many_tiles = qrows / kLargeRows + base.b.seqs;
    hipLaunchKernelGGL((attend_few_kernel<T, D, FMT>),
                       dim3(static_cast<unsigned>(few_tiles * heads + kTargetSmall)), dim3(256),
                       0, s, few);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!only) {
        hipLaunchKernelGGL((attend_many_kernel<T, D, FMT>),
                           dim3(static_cast<unsigned>(many_tiles * heads + kTargetLarge)),
                           dim3(256), 0, s, many);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // (a pair of tile and head with several runs has two at least)
    const uint32_t few_blocks = kSlotsFew / 2;
    const uint32_t many_blocks = only ? 0 : kSlotsMany / 2 * (kLargeRows / kJoinRows);
    hipLaunchKernelGGL((join_kernel<T, D>), dim3(few_blocks + many_blocks), dim3(256), 0, s, few,
                       many, few_blocks);
    return hipGetLastError();
}

template <typename T>
hipError_t attend(const AttArgs &a, char *ws, hipStream_t s) {
    const bool fp4 = a.c.format == TCQ_FP4;
    switch (a.c.dim) {
        case 64:
            return fp4 ? attend<T, 64, TCQ_FP4>(a, ws, s) : attend<T, 64, TCQ_FP8>(a, ws, s);
        case 128:
            return fp4 ? attend<T, 128, TCQ_FP4>(a, ws, s) : attend<T, 128, TCQ_FP8>(a, ws, s);
        default:
            return fp4 ? attend<T, 256, TCQ_FP4>(a, ws, s) : attend<T, 256, TCQ_FP8>(a, ws, s);
    }
}

}  // namespace

size_t attention_bytes(int dim, int heads, int group, int64_t seqs, int64_t rows) {
    (void)heads;
    if (rows == 0 || seqs == 0) return 0;
    size_t n = static_cast<size_t>(kSlotsFew * slot_bytes(kSmallRows, dim));
    if (!few_only(rows, group, seqs))
        n += static_cast<size_t>(kSlotsMany * slot_bytes(kLargeRows, dim));
    return align_up(n, 256);
}

hipError_t launch_attention(const AttentionCall &c, char *ws, hipStream_t s) {
    const double factor = static_cast<double>(c.scale) * 1.44269504088896340736;
    AttArgs a{};
    a.c = c.c;
    a.b = c.b;
    a.q = c.q;
    a.o = c.o;
    a.group = c.group;
    a.rows = c.rows;
    a.factor = static_cast<float>(factor);
    a.factor_low = static_cast<float>(factor - a.factor);
    switch (c.dtype) {
        case TCQ_F32: return attend<float>(a, ws, s);
        case TCQ_F16: return attend<_Float16>(a, ws, s);
        default: return attend<__bf16>(a, ws, s);
    }
}

}  // namespace tcq
