// Attention of new tokens over the paged, quantised cache (tcq_cache_attention):
//     o[i] = sum_j p[i][j] v[j] / sum_j p[i][j],   p[i][j] = exp(scale q[i] . k[j] - m[i])
// over the keys j that row i sees, in one pass over the cache with the running maximum m and sum
// of a softmax.  The group query heads that share a head of keys are rows of the same product, so
// a key is read once for all of them.
//
// Every code times its scale is a bf16 number, so keys and values are multiplied as bf16 with
// exact products and fp32 sums.  q and p are held in terms of bf16 whose sum they are: q exactly,
// in one for bf16, two for fp16 and three for fp32; p in three for fp32 (exact) and in two for
// 16-bit queries (to 2^-15, far below the output's own rounding), but for bf16 queries in the
// larger tiles as one fp16 number (to 2^-11), beside values in fp16: see attend_many.  The sum of
// p is that of the rounded ones.
//
// Scores are computed transposed, S^T = K Q^T: a lane holds four keys of one query row, the same
// row in every instruction, so a row's maximum and sum are the lane's own but for three other
// lanes, and p is in place as the second operand of O^T = V^T P^T.  That product's order of
// keys is the one the lanes hold them in, and V is read across through LDS in the same order.
//
// Work is cut into items (sequence, head, tile of query rows, run of keys) by every workgroup, or
// by a kernel before for many sequences, from the lengths on the device, so that the host need
// not know them: runs are as long as lets about the target number of them remain.  A tile with
// one run writes its outputs, others their share, and a second kernel joins shares in the order
// of the runs.
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
    uint32_t slots;
    int *far;                   // whether attend_far_kernel has work (NULL: it does not come)
    uint32_t *plan;             // see plan_kernel; NULL: workgroups scan the sequences themselves
    int both;                   // tiles of 16 rows serve sequences of up to kFewRows rows only,
                                // larger tiles the others (0: this kernel serves every sequence)
};

// ---------------------------------------------------------------- items

// What a launch of tiles of BQ rows does with a sequence.
struct Sequence {
    uint32_t tiles, units, chunks;
};
constexpr int kUnit = 128;      // keys: runs are whole units
constexpr int kSmallRows = 16;      // query rows of the smaller tiles
// Rows of a sequence that they serve beside the larger ones, which read keys less often but hold
// 128 or 256 rows (16 sequences of 2000 to 8000 keys, 32 query heads over 8, bf16: 32 rows 88 us
// with small tiles, 155 with large; 64 rows 122 and 157; 96 rows 173 and 159).
constexpr int kFewRows = 64;
// About how many runs there are to be, given the tiles' units in all.  A compute unit holds one
// workgroup of the larger tiles and two of the smaller ones: as many runs as fill the card once,
// and of the smaller tiles twice as many where each still has 16 units, for the sequences'
// different lengths (one token of 4 sequences of 2000 to 8000 keys, 8 heads of 128: 24 us with 512,
// 30 with 1024; of 16 of 1000 to 16000: 84 and 77; of 64: 261 and 253; 512 tokens behind 32000: 319
// us with 256, 344 with 512).
constexpr int kTargetSmall = 1024, kTargetLarge = 256;
template <int BQ>
__device__ __forceinline__ uint32_t target(uint64_t units) {
    if (BQ != kSmallRows) return kTargetLarge;
    return units < 16 * (kTargetSmall / 2) ? kTargetSmall / 2 : kTargetSmall;
}

// (rows x group is below 2^28 and lengths below 2^31: 32 bits hold rows, keys and units)
template <int BQ>
__device__ __forceinline__ Sequence sequence(const AttArgs &a, int64_t s) {
    Sequence r{0, 0, 1};
    if (s >= a.b.seqs) return r;
    const cache::Span sp = cache::span_of(a.b, s, a.rows);
    const int64_t n = sp.end - sp.begin;
    if (n <= 0) return r;
    const uint32_t rows = static_cast<uint32_t>(n) * static_cast<uint32_t>(a.group);
    const bool small = rows <= kFewRows;
    if (a.both && small != (BQ == kSmallRows)) return r;
    r.tiles = (rows + BQ - 1) / BQ;
    int64_t keys = sp.first + n;  // the last row sees the keys before this
    const int64_t most = a.b.width << a.c.page_log2;
    keys = keys < 0 ? 0 : (keys < most ? keys : most);
    r.units = static_cast<uint32_t>((keys + kUnit - 1) / kUnit);
    return r;
}

// Running sum over the lanes, of which `n` (uniform) at most are not zero; the last of 64 holds
// all.
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v, int lane, int n) {
    for (int d = 1; d < n; d <<= 1) {
        const uint32_t o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}

// Units per run: the fewest with at most about the target number of runs in all, given the units
// of all tiles of a head.
template <int BQ>
__device__ __forceinline__ uint32_t run_units(const AttArgs &a, uint64_t total) {
    total *= a.c.heads;
    const uint32_t runs = target<BQ>(total);
    uint64_t per = (total + runs - 1) / runs;
    per = per > 1 ? per : 1;
    return static_cast<uint32_t>(per < (1u << 30) ? per : 1u << 30);  // (units are fewer)
}
template <int BQ>
__device__ __forceinline__ uint32_t run_units(const AttArgs &a, int lane) {
    if (__builtin_expect(a.plan != nullptr, 0)) return a.plan[0];
    const Sequence q = sequence<BQ>(a, lane);
    uint64_t total = static_cast<uint64_t>(q.tiles) * q.units;
    // (a wave's first lanes hold everything)
    for (int d = 1; d < a.b.seqs; d <<= 1) total += __shfl_xor(total, d);
    return of_lane(run_units<BQ>(a, total), 0);
}

// Of a sequence: its pairs (tile, head) that have several runs, its items (pair, run) and those
// items that are shares.
struct Counts {
    uint32_t pairs, items, shares;
};
// (A launch has fewer than 2^24 workgroups: counts are cut to 2^25 so that 64 of them fit.)
template <int BQ>
__device__ __forceinline__ Counts counts(const AttArgs &a, Sequence &q, uint32_t per) {
    const auto cut = [](uint64_t v) {
        return v < (1u << 25) ? static_cast<uint32_t>(v) : 1u << 25;
    };
    q.chunks = q.units > per ? (q.units + per - 1) / per : 1;
    const uint64_t pairs = static_cast<uint64_t>(q.tiles) * a.c.heads;
    const uint32_t items = cut(pairs * q.chunks);
    return Counts{q.chunks > 1 ? cut(pairs) : 0, items, q.chunks > 1 ? items : 0};
}

// One of the pairs (tile, head) or items (pair, run of keys) of a launch; uniform in a wave.
struct Item {
    int64_t seq;
    uint32_t tiles, chunks;     // of the sequence
    uint32_t left;              // its number in the sequence
    uint32_t slot;              // number of its share
};
// Item (PAIRS: pair with several runs) `index`, or false past the last.
template <int BQ, bool PAIRS>
__device__ __forceinline__ bool item_of(const AttArgs &a, uint32_t index, uint32_t per, int lane,
                                        Item &it) {
    const int seqs = static_cast<int>(a.b.seqs);
    if (__builtin_expect(a.plan != nullptr, 0)) {
        const uint32_t *pairs = a.plan + 4, *items = pairs + seqs, *shares = items + seqs;
        const uint32_t *to = PAIRS ? pairs : items;
        const int s = static_cast<int>(cache::at_most(to, seqs, index, lane));
        if (s >= seqs) return false;
        Sequence q = sequence<BQ>(a, s);
        const Counts c = counts<BQ>(a, q, per);
        it.seq = s;
        it.tiles = of_lane(q.tiles, 0);
        it.chunks = of_lane(q.chunks, 0);
        it.left = of_lane(index - (to[s] - (PAIRS ? c.pairs : c.items)), 0);
        it.slot = of_lane(shares[s] - c.shares, 0) + it.left;
        return true;
    }
    Sequence q = sequence<BQ>(a, lane);
    const Counts c = counts<BQ>(a, q, per);
    const uint32_t n = PAIRS ? c.pairs : c.items;
    const uint32_t to = wave_prefix(n, lane, seqs);
    if (index >= of_lane(to, seqs - 1)) return false;
    const uint32_t stop = wave_prefix(c.shares, lane, seqs);
    // lanes before the item's
    const int at = __popcll(__ballot(lane < seqs && to <= index));
    it.seq = at;
    it.tiles = of_lane(q.tiles, at);
    it.chunks = of_lane(q.chunks, at);
    it.left = index - of_lane(to - n, at);
    it.slot = of_lane(stop - c.shares, at) + it.left;
    return true;
}

// Batches of more than 64 sequences: a workgroup for each size of tile writes the units of a run
// and, over the sequences, running sums of their counts (cut to 2^31), in which the others search.
// (One token of 256 sequences of 100 to 600 keys, 32 query heads over 8 of 128, 66 us, with scans
// of them all in every workgroup 97; of 1024 240 and 623; of 4096 917 and 7350.)
constexpr int kScanned = 64;
constexpr int kPlanThreads = 1024;
int64_t plan_words(int64_t seqs) { return seqs > kScanned ? 4 + (3 * seqs + 3) / 4 * 4 : 0; }
template <int BQ>
__device__ __forceinline__ void plan(const AttArgs &a) {
    constexpr int kWaves = kPlanThreads / 64;
    __shared__ uint64_t sums[3][kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint64_t total = 0;
    for (int64_t s = tid; s < a.b.seqs; s += kPlanThreads) {
        const Sequence q = sequence<BQ>(a, s);
        total += static_cast<uint64_t>(q.tiles) * q.units;
    }
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
    if (lane == 0) sums[0][wave] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWaves; ++w) total += sums[0][w];
    __syncthreads();
    const uint32_t per = run_units<BQ>(a, total);
    if (tid == 0) a.plan[0] = per;
    uint64_t before[3] = {0, 0, 0};
    for (int64_t s0 = 0; s0 < a.b.seqs; s0 += kPlanThreads) {
        const int64_t s = s0 + tid;
        Sequence q = sequence<BQ>(a, s);
        const Counts c = counts<BQ>(a, q, per);
        uint64_t v[3] = {c.pairs, c.items, c.shares};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t o = __shfl_up(v[k], d);
                if (lane >= d) v[k] += o;
            }
            if (lane == 63) sums[k][wave] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint64_t all = 0;
            for (int w = 0; w < kWaves; ++w) {
                if (w == wave) v[k] += before[k] + all;
                all += sums[k][w];
            }
            before[k] += all;
            if (s < a.b.seqs)
                a.plan[4 + k * a.b.seqs + s] =
                    static_cast<uint32_t>(v[k] < (1u << 31) ? v[k] : 1u << 31);
        }
        __syncthreads();
    }
}
template <int BQ>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(AttArgs few, AttArgs many) {
    if (blockIdx.x == 0)
        plan<kSmallRows>(few);
    else
        plan<BQ>(many);
}

// What a workgroup computes, uniform.  Heads vary fastest, so that those of one sequence go to
// different XCDs and a head's tiles to the same one, then tiles, later ones (more keys) first.
template <int BQ>
struct Tile {
    const int32_t *table;       // the sequence's pages
    int head;
    int64_t row0;               // the call's row of the sequence's first new token
    uint32_t rows;              // query rows of the sequence: group to a token
    uint32_t r0;                // the tile's first
    int first;                  // position of the sequence's first new token
    uint32_t begin, end;        // keys of the run that some row of the tile sees
    uint32_t slot;
    bool share;

    __device__ __forceinline__ bool init(const AttArgs &a, uint32_t index, int lane) {
        const uint32_t per = run_units<BQ>(a, lane);
        Item it;
        if (!item_of<BQ, false>(a, index, per, lane, it)) return false;
        set(a, it);
        share = it.chunks > 1;
        slot = it.slot;
        if (share && slot >= a.slots) return false;
        const uint32_t chunk = it.left / a.c.heads / it.tiles;
        const uint64_t from = static_cast<uint64_t>(chunk) * per * kUnit;
        const uint64_t to = chunk + 1 < it.chunks ? from + static_cast<uint64_t>(per) * kUnit
                                                  : uint64_t{1} << 31;
        const uint32_t last = (r0 + BQ < rows ? r0 + BQ : rows) - 1;
        int64_t keys = static_cast<int64_t>(first) + last / a.group + 1;
        const int64_t most = a.c.pages > 0 ? a.b.width << a.c.page_log2 : 0;
        keys = keys < most ? keys : most;
        keys = keys < static_cast<int64_t>(to) ? keys : static_cast<int64_t>(to);
        begin = static_cast<uint32_t>(from);
        end = keys > 0 ? static_cast<uint32_t>(keys) : 0;
        return true;
    }
    __device__ __forceinline__ void set(const AttArgs &a, const Item &it) {
        const cache::Span sp = cache::span_of(a.b, it.seq, a.rows);
        table = a.b.table + it.seq * a.b.ldt;
        head = static_cast<int>(it.left % a.c.heads);
        r0 = (it.tiles - 1 - it.left / a.c.heads % it.tiles) * BQ;
        row0 = sp.begin;
        rows = static_cast<uint32_t>(sp.end - sp.begin) * static_cast<uint32_t>(a.group);
        // (positions before -2^24 are as good as -2^24: a sequence has at most 2^23 rows)
        first = static_cast<int>(sp.first > -(1 << 24) ? sp.first : -(1 << 24));
    }
    // The last key that query row r sees, -1 for none.
    __device__ __forceinline__ int sees(const AttArgs &a, uint32_t r) const {
        const int64_t p = static_cast<int64_t>(first) + r / a.group;
        return p < 0 ? -1 : (p < INT32_MAX ? static_cast<int>(p) : INT32_MAX);
    }
    // Offset of query row r's vector.
    __device__ __forceinline__ int64_t at(const AttArgs &a, const CacheRows &x, uint32_t r) const {
        const uint32_t i = r / a.group;
        return (row0 + i) * x.row +
               (static_cast<int64_t>(head) * a.group + (r - i * a.group)) * x.head;
    }
};

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

// The same as numbers N: one fp16 number, or bf16 terms.
template <typename N, int TERMS>
__device__ __forceinline__ void numbers_of(float a, float b, uint32_t (&w)[TERMS]) {
    if constexpr (__is_same(N, _Float16)) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        static_assert(TERMS == 1, "one number");
        w[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
    } else {
        terms_of<TERMS>(a, b, w);
    }
}

// Terms of q, and of p in the larger tiles (bf16: see attend_many).
template <typename T>
constexpr int terms() {
    return sizeof(T) == 4 ? 3 : (__is_same(T, _Float16) ? 2 : 1);
}
// Terms of p in the tiles of 16 rows.
template <typename T>
constexpr int few_weight_terms() {
    return sizeof(T) == 4 ? 3 : 2;
}

// One and infinity as bits of a 16-bit type.
template <typename N>
constexpr short kOne = __is_same(N, _Float16) ? 0x3C00 : 0x3F80;
template <typename N>
constexpr short kInf = __is_same(N, _Float16) ? 0x7C00 : 0x7F80;

// One 16 x 16 product over 32 keys or dims, smallest term first.
template <typename N, int TERMS>
__device__ __forceinline__ f32x4 mma_terms(const s16x8 &x, const s16x8 (&y)[TERMS], f32x4 c) {
#pragma unroll
    for (int n = TERMS - 1; n >= 0; --n) c = gemm::Traits<N>::mma(x, y[n], c);
    return c;
}

// f over the four lanes that hold a query row's keys: lanes l, l ^ 16, l ^ 32,
// l ^ 48.  A swap of one register with itself leaves each half's values in all lanes.
template <typename F>
__device__ __forceinline__ float over_row(float v, const F &f) {
    const uint32_t u = __float_as_uint(v);
    const auto halves = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float w = f(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
    const uint32_t t = __float_as_uint(w);
    const auto rows = __builtin_amdgcn_permlane16_swap(t, t, false, false);
    return f(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
}
__device__ __forceinline__ float row_max(float v) {
    return over_row(v, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}
// The largest of N (NaN if one is: the row's outputs are NaN then, whatever the others are taken
// relative to), without the canonicalising moves that fmaxf of a product's sums takes.
template <int N>
__device__ __forceinline__ float largest(const f32x4 (&s)[N / 4]) {
    float top = __builtin_elementwise_maximum(s[0][0], s[0][1]);
#pragma unroll
    for (int i = 2; i < N; i += 2)
        top = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(s[i / 4][i % 4], s[i / 4][i % 4 + 1]), top);
    return top;
}

// The running softmax of one query row per lane.  Weights are taken relative to a score that the
// largest so far exceeds by at most kSlack (powers of two): sums and outputs are rescaled only
// when it grows beyond, not at every tile with a new largest score.
//   The sum is a product with ones, of the weights as they meet the values: their rounding then
// cancels in part, and the sum of a row is in every lane that holds it.
struct Softmax {
    static constexpr float kSlack = 8.0f;
    float top;    // that score times factor, -inf before the first key
    f32x4 sum;    // four times the same
    __device__ __forceinline__ void init() {
        top = -__builtin_inff();
        sum = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    template <typename N, int TERMS>
    __device__ __forceinline__ void add(const s16x8 (&p)[TERMS]) {
        constexpr short o = kOne<N>;
        const s16x8 ones = {o, o, o, o, o, o, o, o};
        sum = mma_terms<N, TERMS>(ones, p, sum);
    }
    static __device__ __forceinline__ float safe(float t) {
        return t == -__builtin_inff() ? 0.0f : t;
    }
    // Takes a tile's largest score (times factor) along; true if anything is to be multiplied by
    // alpha (in some lane).
    __device__ __forceinline__ bool grow(float score, float &alpha) {
        if (!__any(score > top + kSlack)) return false;
        const float to = score > top ? score : top;
        alpha = __builtin_amdgcn_exp2f(top - safe(to));
        top = to;
        sum *= alpha;
        return true;
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

// Tiles in LDS have rows of W bytes (D bf16 numbers) whose pieces are permuted by the low bits of
// the row: a key's 16-byte chunks (read 16 rows at a time) and a value's 32-byte units (read
// across, eight rows at a time).  The permutation is an exclusive or of the offset's bits, so one
// offset per thread and an exclusive or with a constant give every address.
template <int W>
struct Units {
    static constexpr int kMask = W / 32 < 8 ? W / 32 - 1 : 7;
    // Offset of unit 0 of row r; unit u's is it ^ 32 u.
    static __device__ __forceinline__ int row(int r) { return r * W + (r & kMask) * 32; }
    // What lane `lane` reads from to get 32 rows across: columns 16 u .. 16 u + 15 with ^ 32 u.
    static __device__ __forceinline__ int across(int lane) {
        const int l16 = lane & 15;
        return row(4 * (lane >> 4) + (l16 >> 2)) + (l16 & 3) * 8;
    }
};
// A = X^T of 16 columns and 32 rows: row 4 g + i of them in place i and row 16 + 4 g + i in place 4
// + i of lane group g.
template <int W>
__device__ __forceinline__ s16x8 read_across(const char *at) {
    typedef __attribute__((address_space(3))) s16x4 *P;
    s16x8 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(at + h * 16 * W));
#pragma unroll
        for (int v = 0; v < 4; ++v) out[h * 4 + v] = t[v];
    }
    return out;
}

// 16 bytes of codes (16 of fp8, 32 of fp4) to words of two 16-bit numbers.
template <int FMT, typename N = __bf16>
__device__ __forceinline__ void decode16(const u32x4 &q, float s, uint32_t *w) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t *to = w + (FMT == TCQ_FP4 ? 4 : 2) * j;
        if constexpr (__is_same(N, _Float16))
            mx::decode_word_f16<FMT>(q[j], s, to);
        else
            mx::decode_word_bf16<FMT>(q[j], s, to);
    }
}

// Whether some of 16 bytes of codes is not zero.
template <int FMT>
__device__ __forceinline__ bool any_code(const u32x4 &c) {
    constexpr uint32_t kSize = FMT == TCQ_FP4 ? 0x77777777u : 0x7F7F7F7Fu;
    return ((c[0] | c[1] | c[2] | c[3]) & kSize) != 0;
}

// ---------------------------------------------------------------- outputs

// Shares of a tile: BQ x D sums, then BQ maxima and BQ sums of weights.
template <int BQ, int D>
constexpr int64_t slot_floats() {
    return BQ * (D + 2);
}

// Four consecutive outputs d .. d + 3 of query row r of the sequence; a row that saw no key: zeros.
template <typename T, int BQ>
__device__ __forceinline__ void store(const AttArgs &a, const Tile<BQ> &t, uint32_t r, int d, f32x4 o,
                                      float sum) {
    if (r >= t.rows) return;
    const float inv = 1.0f / sum;
    Packed<T, 4> p;
#pragma unroll
    for (int v = 0; v < 4; ++v) p.v[v] = static_cast<T>(sum == 0.0f ? 0.0f : o[v] * inv);
    T *out = static_cast<T *>(const_cast<void *>(a.o.p)) + t.at(a, a.o, r) + d;
    *reinterpret_cast<Packed<T, 4> *>(out) = p;
}

// The same for row r of the tile: as they are (a single run) or into its share.
template <typename T, int BQ, int D>
__device__ __forceinline__ void put(const AttArgs &a, const Tile<BQ> &t, int r, int d, f32x4 o,
                                    float top, float sum) {
    if (!t.share) {
        store<T, BQ>(a, t, t.r0 + r, d, o, sum);
        return;
    }
    float *slot = a.part + t.slot * slot_floats<BQ, D>();
    *reinterpret_cast<f32x4 *>(slot + r * D + d) = o;
    if (d == 0) {
        slot[BQ * D + r] = top;
        slot[BQ * D + BQ + r] = sum;
    }
}

// The fragments of query row `r` (this lane's) in terms: place 8 f + v of lane group g holds d =
// at(f) + v.  An infinity becomes NaN, as the row's outputs are: scores that are all -inf would
// pass for keys that it does not see.  (Terms after the first are NaN by themselves there.)
template <typename T, int D, int TERMS, int BQ, typename At>
__device__ __forceinline__ void load_query(const AttArgs &a, const Tile<BQ> &t, uint32_t r,
                                           const At &at, s16x8 (&q)[TERMS][D / 32]) {
    const bool in = r < t.rows;
    const T *x = static_cast<const T *>(a.q.p) + t.at(a, a.q, in ? r : t.rows - 1);
#pragma unroll
    for (int f = 0; f < D / 32; ++f) {
        const Packed<T> p = *reinterpret_cast<const Packed<T> *>(x + at(f));
        u32x4 w[TERMS];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t t2[TERMS];
            float v0 = in ? static_cast<float>(p.v[2 * k]) : 0.0f;
            float v1 = in ? static_cast<float>(p.v[2 * k + 1]) : 0.0f;
            if constexpr (TERMS == 1) {
                v0 = __builtin_fmaf(v0, 0.0f, v0);
                v1 = __builtin_fmaf(v1, 0.0f, v1);
            }
            terms_of<TERMS>(v0, v1, t2);
#pragma unroll
            for (int n = 0; n < TERMS; ++n) w[n][k] = t2[n];
        }
#pragma unroll
        for (int n = 0; n < TERMS; ++n) q[n][f] = __builtin_bit_cast(s16x8, w[n]);
    }
}

// Cache rows of one head: codes and scale bytes of page p's place i lie at p pages and i rows
// behind the head's first.
struct HeadCache {
    const uint8_t *k, *v, *ke, *ve;
    uint32_t pages;
    uint32_t code_page, scale_page;     // bytes of a page: below 2^30
    int log2;
    uint32_t mask;
};
template <int FMT, int D>
__device__ __forceinline__ HeadCache head_cache(const AttArgs &a, int head) {
    HeadCache h;
    const int64_t row = static_cast<int64_t>(head) << a.c.page_log2;
    h.k = a.c.k_codes + row * mx::bytes<FMT>(D);
    h.v = a.c.v_codes + row * mx::bytes<FMT>(D);
    h.ke = a.c.k_scale + row * (D / 32);
    h.ve = a.c.v_scale + row * (D / 32);
    h.pages = static_cast<uint32_t>(a.c.pages);
    const uint32_t rows = static_cast<uint32_t>(a.c.heads) << a.c.page_log2;
    h.code_page = rows * mx::bytes<FMT>(D);
    h.scale_page = rows * (D / 32);
    h.log2 = a.c.page_log2;
    h.mask = (1u << a.c.page_log2) - 1;
    return h;
}

// acc += x p for a tile of values among which some stand for NaN, where a row does not see every
// key (bit i of sees: the key in the lane's place i): a NaN reaches the rows that see its key,
// whatever p, and no other (0 times NaN would).  The rows it reaches are those whose count of NaN
// keys, the product of ones, is not zero.
template <typename N, int TERMS>
__device__ __forceinline__ void add_wild(const s16x8 &x, const s16x8 (&p)[TERMS], uint32_t sees,
                                         f32x4 &acc) {
    s16x8 clean, nan, ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool bad = (x[i] & 0x7FFF) > kInf<N>;
        clean[i] = bad ? 0 : x[i];
        nan[i] = bad ? kOne<N> : 0;
        ones[i] = sees >> i & 1 ? kOne<N> : 0;
    }
    const f32x4 n = gemm::Traits<N>::mma(nan, ones, f32x4{0.f, 0.f, 0.f, 0.f});
    acc = mma_terms<N, TERMS>(clean, p, acc);
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (n[v] != 0.0f) acc[v] = __builtin_nanf("");
}

// ---------------------------------------------------------------- few query rows

// 16 query rows, four waves that take every fourth tile of 32 keys of the run, each with its own
// softmax; joined in LDS.  Keys go from memory straight into the first operand of S^T (a lane
// reads a run of D / 4 dims of its key), values through the wave's own piece of LDS.  A tile's
// codes are asked for while the one before is multiplied, its page numbers one earlier.
//   Bound to two waves to a SIMD the compiler keeps the outputs out of the accumulation registers,
// whose copies cost a tile 128 instructions (64 sequences, 4 heads of 128: fp32 over fp8 191 us,
// 145 with; bf16 over fp4 99 and 96).  256 dims do not fit but for bf16 over fp4 (235 and 196; fp8
// 305 and 544).
//   Bound by memory: 64 sequences of 1000 to 16000 keys, 8 heads of 128, fp8, 252 us at 4.6 TB/s.
//   So bf16 queries' weights in two terms cost little, and leave the outputs' own rounding alone
// (relative to the norm of float64 outputs 1.66e-3 there, the outputs' rounding itself, and 2.33e-3
// with one term): 252 us with either, 64 sequences over fp4 96 and 94, 256 of 100 to 600 keys 68
// and 67, 16 of 8 tokens 87 and 85, 256 dims over fp4 180 and 171.
template <typename T, int D, int FMT>
constexpr int few_waves() {
    return D < 256 || (FMT == TCQ_FP4 && terms<T>() == 1) ? 2 : 1;
}
template <typename T, int D, int FMT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(few_waves<T, D, FMT>()))) void
attend_few_kernel(AttArgs a) {
    constexpr int TERMS = terms<T>();
    constexpr int PT = few_weight_terms<T>();
    constexpr int BQ = kSmallRows;
    constexpr int kRow = mx::bytes<FMT>(D);    // bytes of a cache row
    constexpr int kRun = kRow / 4;             // of it, one lane's
    constexpr int kKLoads = kRun >= 16 ? kRun / 16 : 1;
    constexpr int kLanes = kRow / 16;          // lanes to a row of values
    constexpr int kPerLoad = 64 / kLanes;      // rows of values to a load
    constexpr int kVLoads = 32 / kPerLoad;
    constexpr int kGroups = D / 32;
    constexpr int kKScales = kGroups > 4 ? 2 : 1;
    constexpr int kTiles = D / 16;             // tiles of 16 dims
    constexpr int kWords = FMT == TCQ_FP4 ? 16 : 8;   // of bf16 pairs in 16 bytes of codes
    __shared__ __align__(16) char lds[4 * 32 * D * 2];
    __shared__ float tops[4][16], sums[4][16];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (a.far && blockIdx.x == 0 && tid == 0) *a.far = 0;  // (before the larger tiles' launch)
    Tile<BQ> tile;
    if (!tile.init(a, blockIdx.x, lane)) return;
    const HeadCache hc = head_cache<FMT, D>(a, tile.head);
    const int seen_by_all = tile.sees(a, tile.r0);
    const int mine = tile.sees(a, tile.r0 + l16);

    char *vt = lds + wave * (32 * D * 2);
    const int part = lane % kLanes;
    // (row j kPerLoad + lane / kLanes, whose low bits j takes part in)
    auto to_lds = [&](int j) {
        return Units<D * 2>::row(j * kPerLoad + lane / kLanes) ^ (part * (kWords / 8) * 32);
    };
    const int from_lds = Units<D * 2>::across(lane);
    // the page of key base + lane % 32 (past the end: the last one's)
    auto find = [&](uint32_t base) {
        const uint32_t pos = base + (lane & 31);
        return tile.table[(pos < tile.end ? pos : tile.end - 1) >> hc.log2];
    };
    struct Codes {
        u32x4 k[2][kKLoads];
        int ke[2][kKScales];
        u32x4 v[kVLoads];
        int ve[kVLoads];
        uint32_t there;      // bit t: key t of the tile is
    };
    // (keys that are not there read the cache's first bytes, and are masked)
    auto load = [&](uint32_t base, int page, Codes &c) {
        const bool whole = hc.log2 >= 5;   // (tiles start on multiples of 32: one page holds one)
        const bool in = static_cast<uint32_t>(page) < hc.pages && base + (lane & 31) < tile.end;
        c.there = static_cast<uint32_t>(__ballot(in));
        page = in ? page : 0;
        const uint32_t all = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(page));
        auto page_at = [&](int t) {
            return whole ? all : static_cast<uint32_t>(__shfl(page, t));
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = 16 * h + l16;
            const uint32_t p = page_at(t), i = (base + t) & hc.mask;
            const uint8_t *x =
                hc.k + static_cast<uint64_t>(p) * hc.code_page + i * kRow + g * kRun;
            const uint8_t *e = hc.ke + static_cast<uint64_t>(p) * hc.scale_page + i * kGroups +
                               (g * (D / 4)) / 32;
#pragma unroll
            for (int j = 0; j < kKLoads; ++j) {
                if constexpr (kRun >= 16) {
                    c.k[h][j] = *reinterpret_cast<const u32x4 *>(x + 16 * j);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(x);
                    c.k[h][j] = u32x4{w.x, w.y, 0, 0};
                }
            }
#pragma unroll
            for (int j = 0; j < kKScales; ++j) c.ke[h][j] = e[j];
        }
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) {
            const int t = j * kPerLoad + lane / kLanes;
            const uint32_t p = page_at(t), i = (base + t) & hc.mask;
            c.v[j] = *reinterpret_cast<const u32x4 *>(
                hc.v + static_cast<uint64_t>(p) * hc.code_page + i * kRow + part * 16);
            c.ve[j] = hc.ve[static_cast<uint64_t>(p) * hc.scale_page + i * kGroups +
                            part / (kLanes / kGroups)];
        }
    };

    uint32_t base = tile.begin + 32 * wave;
    int page = 0;
    Codes now;
    if (tile.begin < tile.end) {
        page = find(base);
        load(base, page, now);
        page = find(base + 128);
    }
    s16x8 q[TERMS][kGroups];
    load_query<T, D, TERMS>(a, tile, tile.r0 + l16, [&](int f) { return g * (D / 4) + 8 * f; }, q);
    f32x4 acc[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    Softmax sm;
    sm.init();
    for (; base < tile.end; base += 128) {
        const uint32_t there = now.there;
        // scores
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0.f, 0.f, 0.f, 0.f};
            uint32_t w[D / 8];
            if constexpr (kRun < 16) {
                mx::decode_word_bf16<FMT>(now.k[h][0][0], mx::scale_of(now.ke[h][0]), w);
                mx::decode_word_bf16<FMT>(now.k[h][0][1], mx::scale_of(now.ke[h][0]), w + 4);
            } else {
                // (16 bytes of fp8 are half a group)
#pragma unroll
                for (int j = 0; j < kKLoads; ++j)
                    decode16<FMT>(now.k[h][j], mx::scale_of(now.ke[h][FMT == TCQ_FP4 ? j : j / 2]),
                                  w + kWords * j);
            }
#pragma unroll
            for (int f = 0; f < kGroups; ++f) {
                const s16x8 x = __builtin_bit_cast(
                    s16x8, (u32x4{w[4 * f], w[4 * f + 1], w[4 * f + 2], w[4 * f + 3]}));
                s16x8 y[TERMS];
#pragma unroll
                for (int n = 0; n < TERMS; ++n) y[n] = q[n][f];
                s[h] = mma_terms<__bf16, TERMS>(x, y, s[h]);
            }
        }
        // values into LDS
        bool wild = false;   // some stand for NaN
#pragma unroll
        for (int j = 0; j < kVLoads; ++j) {
            if (there != 0xFFFFFFFFu && !(there >> (j * kPerLoad + lane / kLanes) & 1)) {
                now.v[j] = u32x4{0, 0, 0, 0};
                now.ve[j] = 127;
            }
            wild |= now.ve[j] == 255;
            uint32_t w[kWords];
            decode16<FMT>(now.v[j], mx::scale_of(now.ve[j]), w);
#pragma unroll
            for (int u = 0; u < kWords / 8; ++u) {
                u32x4 *p = reinterpret_cast<u32x4 *>(
                    vt + (to_lds(j) ^ (u * 32)));
                p[0] = u32x4{w[8 * u], w[8 * u + 1], w[8 * u + 2], w[8 * u + 3]};
                p[1] = u32x4{w[8 * u + 4], w[8 * u + 5], w[8 * u + 6], w[8 * u + 7]};
            }
        }
        load(base + 128, page, now);
        page = find(base + 256);
        // mask: keys that are not there, and those past this lane's row
        uint32_t sees = 0xFFu;  // bit 4 h + v: key 16 h + 4 g + v
        if (there != 0xFFFFFFFFu || static_cast<int64_t>(base) + 31 > seen_by_all) {
            sees = 0;
            const int to = mine - static_cast<int>(base) - 4 * g;
            const uint32_t here = there >> (4 * g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = 16 * (i / 4) + i % 4;
                if ((here >> t & 1) && t <= to) sees |= 1u << i;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(sees >> i & 1)) s[i / 4][i % 4] = -__builtin_inff();
        }
        float alpha;
        if (sm.grow(row_max(largest<8>(s)) * a.factor, alpha)) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) acc[t] *= alpha;
        }
        const float ref = Softmax::safe(sm.top);
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = weight<PT>(s[i / 4][i % 4], a.factor, a.factor_low, ref);
        s16x8 pf[PT];
        {
            u32x4 w[PT];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t t[PT];
                terms_of<PT>(p[2 * k], p[2 * k + 1], t);
#pragma unroll
                for (int n = 0; n < PT; ++n) w[n][k] = t[n];
            }
#pragma unroll
            for (int n = 0; n < PT; ++n) pf[n] = __builtin_bit_cast(s16x8, w[n]);
        }
        sm.add<__bf16>(pf);
        __builtin_amdgcn_wave_barrier();
        if (__builtin_expect(__any(wild) && __any(sees != 0xFFu), 0)) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                add_wild<__bf16, PT>(read_across<D * 2>(vt + (from_lds ^ (t * 32))), pf, sees, acc[t]);
        } else {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                acc[t] = mma_terms<__bf16, PT>(read_across<D * 2>(vt + (from_lds ^ (t * 32))), pf,
                                               acc[t]);
        }
        __builtin_amdgcn_wave_barrier();
    }
    // join the waves
    if (g == 0) {
        tops[wave][l16] = sm.top;
        sums[wave][l16] = sm.sum[0];
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
        put<T, BQ, D>(a, tile, r, d4 * 4, o, top, total);
    }
}

// ---------------------------------------------------------------- many query rows

// NQ tiles of 16 query rows to each of NW waves.  The workgroup's threads decode tiles of keys into
// LDS for all waves: while a tile is multiplied, the next one's codes, which arrived during the
// tile before, go into LDS, and those of the one after are asked for.
//   With eight waves the second four meet the others between their scores and their softmax, the
// first four after the whole tile, so that one wave of a SIMD computes its softmax while the other
// multiplies; values are kept for a tile longer for it.
//   Bound by what two waves of a SIMD issue between two meetings: four chunks of 511 to 2048 tokens
// behind 4000 to 16384, 32 query heads over 8 of 128, bf16, 1290 us (850 TF) with the matrix cores
// busy for 37 % of the clocks, VALU for 43 and LDS for 35.  (Without the third of the latter that
// are bank conflicts of the keys' reads it took 3 % more.)
//   bf16 queries' weights meet the values as one fp16 number each, lifted by 2^7, so to 2^-11 of
// themselves or 2^-32 of the row's largest; values as the fp16 numbers that they are relative to
// the first tile's largest scale byte.  Outputs are then as near float64's as their own rounding
// and one per cent of it (1.67e-3 of their norm, 1.66e-3 with exact weights).  The four chunks
// take 1292 us so, 1242 with weights of one bf16 number (2^-8: 2.34e-3) and 1740 with two; 64
// dims 835, 822 and 998; 256 dims (four chunks of 511 to 1024 behind 4000 to 8192, 16 query heads
// over 4) 603, 632 and 702.  Values whose scale bytes lie further apart than fp16's range:
// attend_far_kernel.
// What a workgroup's threads share.
struct ManyLds {
    char *kt, *vt;      // two tiles of keys, three of values
    // of tile i in place i mod 4: the keys that are not there, whether a value stands for NaN
    unsigned long long *absent_of;
    int *wild_of;
    int *top_of;        // the first tile's largest scale byte
    int *far_of;        // whether a value is far from it
};
template <int D>
constexpr int kManyKeys = D == 256 ? 32 : 64;      // of a tile

// Item `index`, values and weights as numbers N, the weights in PT terms.  False: N is fp16, and
// some value is no fp16 number; nothing is written then.
template <typename T, typename N, int PT, int D, int FMT, int NW, int NQ>
__device__ __forceinline__ bool attend_many(const AttArgs &a, const ManyLds &lds, uint32_t index,
                                            int tid) {
    constexpr int TERMS = terms<T>();
    constexpr bool kHalf = __is_same(N, _Float16);
    constexpr int NT = NW * 64, BQ = NW * NQ * 16;
    constexpr int KT = kManyKeys<D>;
    constexpr int kSub = KT / 16, kPairs = KT / 32;
    constexpr int kRow = mx::bytes<FMT>(D);
    constexpr int kLanes = kRow / 16;
    constexpr int kGroups = D / 32;
    constexpr int kTiles = D / 16;
    constexpr int kPieces = KT * kLanes;                       // of 16 bytes, of a tile
    constexpr int kLoads = (kPieces + NT - 1) / NT;
    constexpr int kWords = FMT == TCQ_FP4 ? 16 : 8;            // of bf16 pairs to a piece
    constexpr int kTileBytes = KT * D * 2;
    // (fp16 weights, at most 2^8 past their reference, are lifted to below 2^15)
    constexpr float kLift = kHalf ? 7.0f : 0.0f;
    char *const kt = lds.kt, *const vt = lds.vt;
    const int lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool late = wave >= 4;
    Tile<BQ> tile;
    if (!tile.init(a, index, lane)) return true;
    const HeadCache hc = head_cache<FMT, D>(a, tile.head);
    const uint32_t r0 = tile.r0 + wave * (NQ * 16);
    const int seen_by_all = tile.sees(a, r0);
    int mine[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) mine[n] = tile.sees(a, r0 + 16 * n + l16);

    // Pieces of this thread: key p / kLanes of a tile, bytes 16 (p % kLanes) of its row.
    const int part = tid % kLanes;
    static_assert(NT % kLanes == 0, "a thread's pieces are the same part of their rows");
    int32_t page[kLoads];   // of the keys to be asked for next
    auto find = [&](uint32_t base) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t pos = base + (j * NT + tid) / kLanes;
            page[j] = tile.table[(pos < tile.end ? pos : tile.end - 1) >> hc.log2];
        }
    };
    // A wave's pieces of one turn are 64 / kLanes neighbouring keys: of one page, unless pages are
    // smaller.
    constexpr int kTogether = 64 / kLanes;
    const bool whole = (1u << hc.log2) >= kTogether;
    struct Codes {
        u32x4 k[kLoads], v[kLoads];
        int ke[kLoads], ve[kLoads];
        uint32_t there;     // bit j
    } now;
    // (keys that are not there read the cache's first bytes, and are masked)
    auto load = [&](uint32_t base) {
        now.there = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t pos = base + (j * NT + tid) / kLanes;
            const bool mine = pos < tile.end && (kPieces % NT == 0 || tid < kPieces);
            const uint32_t i = pos & hc.mask;
            const uint32_t at = i * kRow + part * 16;
            const uint32_t e = i * kGroups + part / (kLanes / kGroups);
            if (whole) {
                const uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(page[j]));
                const bool in = p < hc.pages;
                const uint64_t code = in ? static_cast<uint64_t>(p) * hc.code_page : 0;
                const uint64_t scale = in ? static_cast<uint64_t>(p) * hc.scale_page : 0;
                if (in && mine) now.there |= 1u << j;
                now.k[j] = *reinterpret_cast<const u32x4 *>(hc.k + code + at);
                now.v[j] = *reinterpret_cast<const u32x4 *>(hc.v + code + at);
                now.ke[j] = (hc.ke + scale)[e];
                now.ve[j] = (hc.ve + scale)[e];
            } else {
                uint32_t p = static_cast<uint32_t>(page[j]);
                if (p < hc.pages && mine)
                    now.there |= 1u << j;
                else
                    p = 0;
                const uint64_t code = static_cast<uint64_t>(p) * hc.code_page;
                const uint64_t scale = static_cast<uint64_t>(p) * hc.scale_page;
                now.k[j] = *reinterpret_cast<const u32x4 *>(hc.k + code + at);
                now.v[j] = *reinterpret_cast<const u32x4 *>(hc.v + code + at);
                now.ke[j] = hc.ke[scale + e];
                now.ve[j] = hc.ve[scale + e];
            }
        }
    };
    const int row = tid / kLanes;   // of the first piece; the others are 8 n rows further
    static_assert(NT / kLanes % 8 == 0, "and of the same permutation");
    const int k_to = row * (D * 2) + ((part * (kWords / 4)) ^ (row & 7)) * 16;
    const int v_to = Units<D * 2>::row(row) ^ (part * (kWords / 8) * 32);
    const int k_from = l16 * (D * 2) + (g ^ (l16 & 7)) * 16;
    const int v_from = Units<D * 2>::across(lane);

    s16x8 q[NQ][TERMS][kGroups];
    f32x4 acc[NQ][kTiles];
    Softmax sm[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        sm[n].init();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    int ref = 127;   // values are taken times 2^(127 - ref)
    // The values at hand of piece j into LDS.
    auto put_values = [&](int j, float scale, int v_at) {
        char *v = vt + v_at + j * (NT / kLanes) * (D * 2);
        uint32_t w[kWords];
        decode16<FMT, N>(now.v[j], scale, w);
#pragma unroll
        for (int u = 0; u < kWords / 8; ++u) {
            u32x4 *d = reinterpret_cast<u32x4 *>(v + (v_to ^ (u * 32)));
            d[0] = u32x4{w[8 * u], w[8 * u + 1], w[8 * u + 2], w[8 * u + 3]};
            d[1] = u32x4{w[8 * u + 4], w[8 * u + 5], w[8 * u + 6], w[8 * u + 7]};
        }
    };
    // The codes at hand, tile i's, into LDS.
    auto stage = [&](int k_at, int v_at, int i) {
        bool rare = false;   // values that stand for NaN, or far from the first tile's
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (kPieces % NT == 0 || tid < kPieces) {
                if (!(now.there >> j & 1)) {
                    now.v[j] = u32x4{0, 0, 0, 0};
                    now.ve[j] = 127;
                    atomicOr(&lds.absent_of[i & 3], 1ull << (row + j * (NT / kLanes)));
                }
                char *k = kt + k_at + j * (NT / kLanes) * (D * 2);
                uint32_t w[kWords];
                decode16<FMT>(now.k[j], mx::scale_of(now.ke[j]), w);
#pragma unroll
                for (int u = 0; u < kWords / 4; ++u)
                    *reinterpret_cast<u32x4 *>(k + (k_to ^ (u * 16))) =
                        u32x4{w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]};
                const int e = now.ve[j] - (kHalf ? ref - 127 : 0);
                rare |= kHalf ? static_cast<uint32_t>(e - 127 - mx::kLowF16<FMT>) >
                                    mx::kHighF16<FMT> - mx::kLowF16<FMT>
                              : e == 255;
                put_values(j, mx::scale_of(e), v_at);
            }
        }
        if (!__any(rare)) return;
        if constexpr (kHalf) {
            // Codes of zero are that whatever the scale (but one that stands for NaN): heads padded
            // with zeros come here in every tile.
            rare = false;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int by = now.ve[j] - ref;
                const bool none =
                    !any_code<FMT>(now.v[j]) && now.ve[j] != 255 && (by & 255) != 128;
                rare |= (by < mx::kLowF16<FMT> || by > mx::kHighF16<FMT>) && !none;
            }
        }
        if (__builtin_expect(__any(rare), 0)) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                if (kPieces % NT != 0 && tid >= kPieces) continue;
                const int e = now.ve[j], by = e - ref;
                if (e == 255) lds.wild_of[i & 3] = 1;
                if constexpr (kHalf) {
                    if (by >= mx::kLowF16<FMT> && by <= mx::kHighF16<FMT>) continue;
                    if (e != 255 && any_code<FMT>(now.v[j])) *lds.far_of = 1;
                    put_values(j, mx::scale_of(e == 255 ? 255 : 127), v_at);
                }
            }
        }
    };

    if (tid < 4) lds.absent_of[tid] = 0, lds.wild_of[tid] = 0;
    if (kHalf && tid == 0) *lds.top_of = 0, *lds.far_of = 0;
    uint32_t base = tile.begin;
    if (base < tile.end) {
        find(base);
        load(base);
        find(base + KT);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
        load_query<T, D, TERMS>(a, tile, r0 + 16 * n + l16,
                                [&](int f) { return 32 * f + 8 * g; }, q[n]);
    __syncthreads();
    if (kHalf) {
        if (base < tile.end) {
            int top = 0;
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                if ((now.there >> j & 1) && now.ve[j] != 255 && now.ve[j] > top &&
                    any_code<FMT>(now.v[j]))
                    top = now.ve[j];
            for (int d = 32; d; d >>= 1) {
                const int o = __shfl_xor(top, d);
                top = top > o ? top : o;
            }
            if (lane == 0) atomicMax(lds.top_of, top);
        }
        __syncthreads();
        // (values of zero say nothing: as for a largest one of 2)
        ref = __builtin_amdgcn_readfirstlane(*lds.top_of);
        ref = ref ? ref : (FMT == TCQ_FP4 ? 126 : 120);
    }
    if (base < tile.end) {
        stage(0, 0, 0);
        load(base + KT);
        find(base + 2 * KT);
    }
    __syncthreads();
    // Tile i is staged before meeting i - 1.  After meeting i the early waves are done with it,
    // the late ones have its scores alone, so its keys may be overwritten (by tile i + 2) then,
    // its values (by tile i + 3) and marks after meeting i + 1.
    int v_now = 0, v_next = kTileBytes, v_last = 2 * kTileBytes;
    for (int i = 0; base < tile.end; base += KT, ++i) {
        const int k_now = i & 1 ? kTileBytes : 0;
        if (tid == 0) lds.absent_of[(i + 2) & 3] = 0, lds.wild_of[(i + 2) & 3] = 0;
        __builtin_amdgcn_s_setprio(1);
        // scores
        f32x4 s[NQ][kSub];
#pragma unroll
        for (int h = 0; h < kSub; ++h) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int f = 0; f < kGroups; ++f) {
                const s16x8 x = *reinterpret_cast<const s16x8 *>(
                    kt + ((k_now + k_from) ^ (f * 64)) + 16 * h * (D * 2));
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    s16x8 y[TERMS];
#pragma unroll
                    for (int m = 0; m < TERMS; ++m) y[m] = q[n][m][f];
                    s[n][h] = mma_terms<__bf16, TERMS>(x, y, s[n][h]);
                }
            }
        }
        __builtin_amdgcn_s_setprio(0);
        stage(kTileBytes - k_now, v_next, i + 1);
        load(base + 2 * KT);
        find(base + 3 * KT);
        if (late) __syncthreads();
        const uint64_t absent = lds.absent_of[i & 3];
        const bool wild = lds.wild_of[i & 3] != 0;
        s16x8 pf[NQ][kPairs][PT];
        uint32_t sees[NQ];
        const bool partial = absent != 0 || static_cast<int64_t>(base) + KT - 1 > seen_by_all;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            sees[n] = ~0u;  // bit 4 h + v: key 16 h + 4 g + v
            if (partial) {
                sees[n] = 0;
                const int to = mine[n] - static_cast<int>(base) - 4 * g;
                const uint64_t gone = absent >> (4 * g);
#pragma unroll
                for (int i = 0; i < 4 * kSub; ++i) {
                    const int t = 16 * (i / 4) + i % 4;
                    if (!(gone >> t & 1) && t <= to) sees[n] |= 1u << i;
                }
#pragma unroll
                for (int i = 0; i < 4 * kSub; ++i)
                    if (!(sees[n] >> i & 1)) s[n][i / 4][i % 4] = -__builtin_inff();
            }
            float alpha;
            const float most = row_max(largest<4 * kSub>(s[n]));
            if (sm[n].grow(kHalf ? __builtin_fmaf(most, a.factor, -kLift) : most * a.factor,
                           alpha)) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) acc[n][t] *= alpha;
            }
            const float top = Softmax::safe(sm[n].top);
            float p[4 * kSub];
#pragma unroll
            for (int i = 0; i < 4 * kSub; ++i)
                p[i] = weight<PT>(s[n][i / 4][i % 4], a.factor, a.factor_low, top);
#pragma unroll
            for (int k2 = 0; k2 < kPairs; ++k2) {
                u32x4 w[PT];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t t[PT];
                    numbers_of<N, PT>(p[8 * k2 + 2 * k], p[8 * k2 + 2 * k + 1], t);
#pragma unroll
                    for (int m = 0; m < PT; ++m) w[m][k] = t[m];
                }
#pragma unroll
                for (int m = 0; m < PT; ++m) pf[n][k2][m] = __builtin_bit_cast(s16x8, w[m]);
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k2 = 0; k2 < kPairs; ++k2) sm[n].template add<N>(pf[n][k2]);
        const auto value = [&](int t, int k2) {
            return read_across<D * 2>(vt + ((v_now + v_from) ^ (t * 32)) + 32 * k2 * (D * 2));
        };
        if (__builtin_expect(wild && partial, 0)) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int k2 = 0; k2 < kPairs; ++k2)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        add_wild<N, PT>(value(t, k2), pf[n][k2], sees[n] >> (8 * k2),
                                        acc[n][t]);
        } else {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
#pragma unroll
                for (int k2 = 0; k2 < kPairs; ++k2) {
                    const s16x8 x = value(t, k2);
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        acc[n][t] = mma_terms<N, PT>(x, pf[n][k2], acc[n][t]);
                }
            }
            __builtin_amdgcn_s_setprio(0);
        }
        if (!late) __syncthreads();
        const int v = v_last;
        v_last = v_now;
        v_now = v_next;
        v_next = v;
    }
    // (every tile was staged before the last meeting)
    if (kHalf && __builtin_expect(*lds.far_of != 0, 0)) return false;
    if constexpr (kHalf) {
        // (the lift leaves sums and outputs alike)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            sm[n].sum[0] *= 0x1p-7f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[n][t][v] = __builtin_amdgcn_ldexpf(acc[n][t][v], ref - 127 - 7);
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            put<T, BQ, D>(a, tile, wave * (NQ * 16) + 16 * n + l16, 16 * t + 4 * g, acc[n][t],
                          sm[n].top, sm[n].sum[0]);
    return true;
}

template <typename T, int D>
constexpr int many_waves() {
    return D == 64 && sizeof(T) == 2 ? 4 : 2;
}
#define TCQ_MANY_LDS                                                                          \
    constexpr int kTileBytes = kManyKeys<D> * D * 2;                                          \
    __shared__ __align__(16) char kt[2 * kTileBytes];                                         \
    __shared__ __align__(16) char vt[3 * kTileBytes];                                         \
    __shared__ unsigned long long absent_of[4];                                               \
    __shared__ int wild_of[4];                                                                \
    __shared__ int top_of, far_of;                                                            \
    const ManyLds lds{kt, vt, absent_of, wild_of, &top_of, &far_of}
template <typename T, int D, int FMT, int NW, int NQ>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(many_waves<T, D>()))) void
attend_many_kernel(AttArgs a) {
    TCQ_MANY_LDS;
    if constexpr (terms<T>() == 1) {
        if (!attend_many<T, _Float16, 1, D, FMT, NW, NQ>(a, lds, blockIdx.x, threadIdx.x) &&
            threadIdx.x == 0)
            *a.far = 1;
    } else {
        attend_many<T, __bf16, terms<T>(), D, FMT, NW, NQ>(a, lds, blockIdx.x, threadIdx.x);
    }
}
// All items again with bf16 values and weights of two terms, where a workgroup met values far
// from one another (the four chunks then take 3350 us), otherwise nothing (2 us).  As another half
// of attend_many_kernel it cost that one up to 9 %, by the order that its loop got.
template <typename T, int D, int FMT, int NW, int NQ>
__global__ __launch_bounds__(NW * 64) void attend_far_kernel(AttArgs a, uint32_t items) {
    TCQ_MANY_LDS;
    if (*a.far == 0) return;
    for (uint32_t i = blockIdx.x; i < items; i += gridDim.x) {
        attend_many<T, __bf16, 2, D, FMT, NW, NQ>(a, lds, i, threadIdx.x);
        __syncthreads();
    }
}
#undef TCQ_MANY_LDS

// ---------------------------------------------------------------- join of shares

// Rows of tiles with several runs.  D / 4 lanes take a row, four dims each; the four waves every
// fourth run, eight at a time (their loads are on their way together), and their sums, each
// relative to the wave's own largest score, are joined in the waves' order.  3.8 us for one token
// of 8 heads of 64, 9.2 for 64 tokens of 32 heads of 128 with 1024 runs.
constexpr int kJoinRows = 16;    // rows to a workgroup
template <typename T, int D, int BQ>
__device__ __forceinline__ void join(const AttArgs &a, uint32_t block) {
    constexpr int kParts = BQ / kJoinRows;
    constexpr int kRows = 256 / D;     // at a time
    constexpr int kBatch = 8;
    __shared__ f32x4 sums[4][64];
    __shared__ float tops[4][64], totals[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Item it;
    const uint32_t per = run_units<BQ>(a, lane);
    if (!item_of<BQ, true>(a, block / kParts, per, lane, it)) return;
    Tile<BQ> tile;
    tile.set(a, it);
    // a pair's shares: one run's are a sequence's pairs apart
    const uint32_t pairs = it.tiles * a.c.heads;
    if (it.slot + static_cast<uint64_t>(it.chunks - 1) * pairs >= a.slots) return;
    const float *slot = a.part + it.slot * slot_floats<BQ, D>();
    const int64_t step = pairs * slot_floats<BQ, D>();
    const int d = lane % (D / 4) * 4;
    const int first = static_cast<int>(block % kParts) * kJoinRows;
    for (int i = 0; i < kJoinRows && tile.r0 + first + i < tile.rows; i += kRows) {
        const int r = first + i + lane / (D / 4);
        float top = -__builtin_inff(), total = 0.0f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (uint32_t c0 = wave; c0 < it.chunks; c0 += 4 * kBatch) {
            float m[kBatch], l[kBatch];
            f32x4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t c = c0 + 4 * k;
                const float *p = slot + (c < it.chunks ? c : c0) * step;
                m[k] = p[BQ * D + r];
                l[k] = p[BQ * D + BQ + r];
                v[k] = *reinterpret_cast<const f32x4 *>(p + r * D + d);
                if (c >= it.chunks) m[k] = -__builtin_inff();
            }
            float to = top;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) to = __builtin_fmaxf(to, m[k]);
            const float ref = Softmax::safe(to);
            const float alpha = __builtin_amdgcn_exp2f(top - ref);
            top = to;
            total *= alpha;
            o *= alpha;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (c0 + 4 * k < it.chunks) {  // (the others are repeats)
                    const float f = __builtin_amdgcn_exp2f(m[k] - ref);
                    total = __builtin_fmaf(l[k], f, total);
                    o += v[k] * f;
                }
            }
        }
        sums[wave][lane] = o;
        tops[wave][lane] = top;
        totals[wave][lane] = total;
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < 4; ++w) top = __builtin_fmaxf(top, tops[w][lane]);
            const float ref = Softmax::safe(top);
            total = 0.0f;
            o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = __builtin_amdgcn_exp2f(tops[w][lane] - ref);
                total = __builtin_fmaf(totals[w][lane], f, total);
                o += sums[w][lane] * f;
            }
            store<T, BQ>(a, tile, tile.r0 + r, d, o, total);
        }
        __syncthreads();
    }
}
template <typename T, int D, int BQ>
__global__ __launch_bounds__(256) void join_kernel(AttArgs few, AttArgs many, uint32_t blocks_few) {
    if (blockIdx.x < blocks_few)
        join<T, D, kSmallRows>(few, blockIdx.x);
    else
        join<T, D, BQ>(many, blockIdx.x - blocks_few);
}

// ---------------------------------------------------------------- host side

// Batches of few rows to a sequence (on average up to 16) are all given to the kernel of 16 rows,
// which saves the other's launch (us so / with both, 4 query heads to each of 8 of 128, bf16): 64
// sequences of 4 tokens behind 4000 130 / 139, 256 of 3 behind 2000 220 / 231, 256 of one behind
// 4000 390 / 399.  A chunk among them is not seen: of 512 tokens behind 2000 among 300 of one token
// 159 / 163, of 512 behind 4000 among 256 491 / 477, of 190 among 64 217 / 191, of 2048 among 700
// of 1000 keys 672 / 522.
bool few_only(int64_t rows, int group, int64_t seqs) {
    return rows * group <= kSmallRows * seqs;
}

// Shares: a sequence has several runs only where they are whole runs of about total / target
// units, so there are at most twice the target.
constexpr int kSlotsFew = 2 * kTargetSmall, kSlotsMany = 2 * kTargetLarge;

constexpr int kLeastRows = 128, kMostRows = 256;   // of a larger tile
constexpr int kManyThreads = 512;                  // and its threads
constexpr uint32_t kFarGrid = 512;
int64_t slot_bytes(int bq, int dim) { return int64_t{bq} * (dim + 2) * 4; }

// Of the shares, a multiple of 16.
int64_t parts_bytes(int dim, bool few) {
    const int64_t n = kSlotsFew * slot_bytes(kSmallRows, dim);
    return few ? n : n + kSlotsMany * slot_bytes(kMostRows, dim);
}

template <typename T, int D, int FMT, int NW, int NQ>
hipError_t attend_as(const AttArgs &base, char *ws, hipStream_t s) {
    constexpr int kRows = NW * NQ * 16;
    static_assert(kRows >= kLeastRows && kRows <= kMostRows && NW * 64 == kManyThreads, "a tile");
    AttArgs few = base, many = base;
    const bool only = few_only(base.rows, base.group, base.b.seqs);
    const int64_t heads = base.c.heads;
    few.both = many.both = !only;
    few.part = reinterpret_cast<float *>(ws);
    few.slots = kSlotsFew;
    many.part = reinterpret_cast<float *>(ws + int64_t{kSlotsFew} * slot_bytes(kSmallRows, D));
    if (base.b.seqs > kScanned) {
        const int64_t words = plan_words(base.b.seqs);
        few.plan = reinterpret_cast<uint32_t *>(ws + parts_bytes(D, only));
        many.plan = few.plan + words;
        hipLaunchKernelGGL((plan_kernel<kRows>), dim3(only ? 1 : 2), dim3(kPlanThreads), 0, s, few,
                           many);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    many.slots = kSlotsMany;
    constexpr bool kFar = terms<T>() == 1;
    if (kFar && !only)
        few.far = many.far =
            reinterpret_cast<int *>(ws + parts_bytes(D, only) + 8 * plan_words(base.b.seqs));
    // tiles of all sequences: whole ones of the rows, and a part of one for each
    const int64_t qrows = base.rows * base.group;
    const int64_t few_tiles = qrows / kSmallRows + base.b.seqs;
    const int64_t few_most = only ? few_tiles : base.b.seqs * (kFewRows / kSmallRows);
    const int64_t tiles = few_tiles < few_most ? few_tiles : few_most;
    const int64_t many_tiles = qrows / kRows + base.b.seqs;
    hipLaunchKernelGGL((attend_few_kernel<T, D, FMT>),
                       dim3(static_cast<unsigned>(tiles * heads + kTargetSmall)), dim3(256), 0, s,
                       few);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!only) {
        hipLaunchKernelGGL((attend_many_kernel<T, D, FMT, NW, NQ>),
                           dim3(static_cast<unsigned>(many_tiles * heads + kTargetLarge)),
                           dim3(NW * 64), 0, s, many);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if constexpr (kFar) {
            const uint32_t items = static_cast<uint32_t>(many_tiles * heads + kTargetLarge);
            hipLaunchKernelGGL((attend_far_kernel<T, D, FMT, NW, NQ>),
                               dim3(items < kFarGrid ? items : kFarGrid), dim3(NW * 64), 0, s,
                               many, items);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    // (a pair of tile and head with several runs has two at least)
    const auto blocks = [&](int64_t n, int slots, int rows) {
        const int64_t pairs = n * heads < slots / 2 ? n * heads : slots / 2;
        return static_cast<uint32_t>(pairs * (rows / kJoinRows));
    };
    const uint32_t few_blocks = blocks(tiles, kSlotsFew, kSmallRows);
    const uint32_t many_blocks = only ? 0 : blocks(many_tiles, kSlotsMany, kRows);
    hipLaunchKernelGGL((join_kernel<T, D, kRows>), dim3(few_blocks + many_blocks), dim3(256), 0, s,
                       few, many, few_blocks);
    return hipGetLastError();
}

// Two tiles of query rows to a wave read a key from LDS half as often as one, but their outputs,
// queries and scores need room, and sequences of up to 256 rows leave half of them idle.  us with
// two / with one (four chunks of 511 to 2048 tokens behind 4000 to 16384, 32 query heads over 8):
//   64 dims: bf16 972 / 839, fp16 1206 / 1186, fp32 2039 / 1704;
//   128 dims: bf16 1289 / 1605, fp16 (spills) 2623 / 2060; 256 dims spill;
//   16 sequences of 256 rows, 128 dims, bf16, 229 both, of 400 rows 331 / 357.
template <typename T, int D, int FMT>
hipError_t attend(const AttArgs &a, char *ws, hipStream_t s) {
    constexpr bool kTwo = D == 128 && terms<T>() == 1;
    if constexpr (kTwo) {
        if (a.rows * a.group > 256 * a.b.seqs) return attend_as<T, D, FMT, 8, 2>(a, ws, s);
    }
    return attend_as<T, D, FMT, 8, 1>(a, ws, s);
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

size_t attention_bytes(int dim, int group, int64_t seqs, int64_t rows) {
    if (rows == 0 || seqs == 0) return 0;
    const bool few = few_only(rows, group, seqs);
    const int64_t n = parts_bytes(dim, few) + 8 * plan_words(seqs) + (few ? 0 : sizeof(int));
    return align_up(static_cast<size_t>(n), 256);
}

size_t attention_most_bytes(int dim, int group, int64_t seqs, int64_t rows) {
    if (rows == 0 || seqs == 0) return 0;
    // (the same rows may come in one sequence)
    const bool few = few_only(rows, group, 1);
    const int64_t n = parts_bytes(dim, few) + 8 * plan_words(seqs) + (few ? 0 : sizeof(int));
    return align_up(static_cast<size_t>(n), 256);
}

int64_t attention_threads(int group, int heads, int64_t seqs, int64_t rows) {
    if (few_only(rows, group, seqs)) return 0;
    return ((rows * group / kLeastRows + seqs) * heads + kTargetLarge) * kManyThreads;
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
