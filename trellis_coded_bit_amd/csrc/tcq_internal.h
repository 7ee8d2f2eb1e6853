// Internal declarations shared by the sources of libtcq (not part of the ABI).
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

namespace tcq {

// Shape of one encode problem after validation.
struct Problem {
    int L, k, V, T;
    int kv;            // k * V: fresh bits per step
    int n;             // steps per block, T / V
    int64_t M, N;
    int64_t ldw;
    int64_t blocks_per_row;
    int64_t nblocks;
    int64_t ngroups;   // 2^(L - kv)
    int64_t nstates;   // 2^L
};

// Workspace plan for one kernel family: per-block bytes, fixed bytes.
struct Plan {
    int variant;              // see kernels
    size_t per_block;         // bytes per block in flight
    size_t fixed;             // bytes independent of the batch size
    size_t bp_bytes;          // backpointer bytes per block
    size_t cost_bytes;        // global cost-vector bytes per block (0: on chip)
};

enum Variant : int {
    kGenericLds = 0,     // any supported shape, cost vectors double-buffered in LDS
    kGenericGlobal = 1,  // any supported shape, cost vectors in the workspace (L2)
    kL16Regs = 2,        // L = 16, k*V = 2, costs in VGPRs (three-step super-steps)
    kL16RegsK3 = 3,      // L = 16, k*V = 3, costs in VGPRs (two-step super-steps)
    kL16RegsHalf = 4,    // L = 16, k*V = 4 (V = 1, 2), run as 2-bit half-steps in VGPRs
};

Plan plan_for(const Problem &p);

// The encoder behind tcq_encode / tcq_encode_timed (tcq_api.cpp): checks the arguments,
// plans the batches for the given workspace and enqueues every kernel.  `fn` names the
// entry point in error messages.  It allocates nothing.
int encode_impl(const char *fn, const float *W, int64_t M, int64_t N, int64_t ldw,
                const float *d, const float *codebook, int L, int k, int V, int T,
                uint32_t *bitstream, uint32_t *start_state, float *cost, float *recon,
                int64_t ldr, void *workspace, size_t workspace_bytes, hipStream_t stream,
                hipEvent_t acs_begin, hipEvent_t acs_end);

// Per-thread error message of the C ABI (tcq_last_error).
void set_error(const char *fmt, ...);
void clear_error();

// Checks shared by the entry points; each returns a status and sets the error message.
int check_trellis(const char *fn, int64_t M, int64_t N, int L, int k, int V, int T);
int check_workspace_alignment(const char *fn, const void *workspace);
int hip_fail(const char *fn, const char *what, hipError_t e);

// Kernel launchers (return hipError_t of the launch).
hipError_t launch_acs_generic(const Problem &p, const Plan &pl, const float *W,
                              const float *d, const float *C, int64_t block0, int64_t nb,
                              char *ws, float *cost, hipStream_t s);
hipError_t launch_traceback_planes(const Problem &p, const Plan &pl, int64_t block0,
                                   int64_t nb, const char *ws, uint32_t *bitstream,
                                   uint32_t *start_state, hipStream_t s);
hipError_t launch_decode(const uint32_t *bitstream, const uint32_t *start_state,
                         const float *C, int64_t M, int64_t N, int L, int k, int V, int T,
                         float *out, int64_t ldo, hipStream_t s);

// Codebook-stream probe of the L = 16 forward kernel (measurement only).
size_t l16_stream_probe_bytes(int64_t blocks);
hipError_t launch_l16_stream_probe(int64_t blocks, int super_steps, char *ws, hipStream_t s);

hipError_t launch_decode_gemv(const uint32_t *bitstream, const uint32_t *start_state,
                              const float *C, const float *x, float *y, int64_t M, int64_t N,
                              int L, int k, int V, int T, hipStream_t s);

// Soft trellis (BCJR).
constexpr int kBcjrMaxKV = 4;                    // 2^kv terms per group kept in registers
constexpr size_t kBcjrLdsBytes = size_t{128} << 10;  // two group vectors in LDS up to this
bool bcjr_supported(int L, int kv);
bool bcjr_in_lds(int L, int kv);
size_t bcjr_per_block_bytes(int L, int kv, int n);
hipError_t launch_bcjr(const float *W, int64_t ldw, const float *d, const float *C, int L, int k,
                       int V, int T, int64_t blocks_per_row, int64_t block0, int64_t nb,
                       float tau, char *ws, float *soft, int64_t ldo, float *logz,
                       hipStream_t s);

// Pre-processing: randomized Hadamard rotation and factored scale field.
constexpr int64_t kHadamardMaxN = 4096;          // longest chunk of the wave kernel
constexpr int64_t kHadamardSmallMaxLen = 8192;   // row length limit when n < 64
hipError_t launch_hadamard(const float *X, int64_t ldx, float *Y, int64_t ldy, int64_t rows,
                           int64_t len, int64_t n, const float *sigma, int inverse,
                           hipStream_t s);
size_t scale_field_slabs(int64_t M);
hipError_t launch_scale_field(const float *W, int64_t ldw, int64_t M, int64_t N, float *a,
                              float *b, float *Wn, int64_t ldn, float *part, hipStream_t s);

// The coded linear layer and its gradients.
struct CodedMatrix {
    const uint32_t *bits, *s0;
    const void *table;       // 2^L x V entries of the layer's type
    int64_t M, N;
    int L, k, V, T;
};
struct LinearCall {
    int dtype, act;
    const void *x;
    int64_t B, ldx;
    const float *row_scale, *bias;
    const void *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
    void *pre;
    int64_t ldp;
};
struct LinearGrad {
    int dtype, act;
    const void *dy;
    int64_t B, lddy;
    const float *row_scale;
    const int8_t *zq;        // checkpoint of the pre-activation: codes, scale bytes
    int64_t ldz;
    const uint8_t *ze;
    const int8_t *xq;        // checkpoint of the input
    int64_t ldxq;
    const uint8_t *xe;
    void *dx;
    int64_t lddx;
    void *dw;
    int64_t lddw;
    float *dbias;
};
// How a product is laid out: tile, steps of k, and how many workgroups share a tile's steps
// (their fp32 shares, part_bytes in all, have rows of part_ld values).
enum GemmTile : int { kTile64 = 0, kTile128 = 1, kTile256 = 2 };
struct GemmPlan {
    int tile, splits, steps, steps_per_split;
    int64_t part_ld;
    size_t part_bytes;
};
GemmPlan gemm_plan(size_t size, int64_t I, int64_t J, int64_t K, int terms);
// Workspace of a call: byte offsets of the decoded matrix (M x ldn), the staged or unpacked
// input rows (B x ldn), the scaled gradient's terms (B x ldm each) and the row scale's
// largest value, the bias gradient's partial sums and the products' shares.
struct LinearLayout {
    size_t matrix, rows, grad, low, tops, part, sums, bytes;
    int64_t ldn, ldm;
    GemmPlan forward, dx, dw;
};
// Batch tiles of 16 rows that a forward call takes at a time with the matrix decoded inside
// the product, or 0 where it is decoded into the workspace first.
int linear_small(size_t size, int64_t B, int64_t N, int L, int k, int V, int T);
size_t linear_small_bytes(size_t size, int64_t N, int bt);
LinearLayout linear_layout(size_t size, int64_t B, int64_t M, int64_t N);
LinearLayout linear_grad_layout(size_t size, int64_t B, int64_t M, int64_t N, bool dx, bool dw,
                                bool dbias, int terms);
hipError_t launch_linear(const CodedMatrix &w, const LinearCall &c, char *ws, hipStream_t s);
hipError_t launch_linear_grad(const CodedMatrix &w, const LinearGrad &c, char *ws,
                              hipStream_t s);

// Products of dense matrices with the tiles of the coded linear layer.
//   bf16 x (B x K) and w (M x K), K a multiple of 8, rows of whole 16-byte pieces:
//   y = x w^T + bias + residual in `dtype`; ws holds gemm_shares(2, B, M, K, 1) bytes.
struct DenseProduct {
    const uint16_t *x, *w;
    int64_t ldx, ldw, B, M, K;
    int dtype;
    const float *bias;
    const void *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
};
size_t gemm_shares(size_t size, int64_t I, int64_t J, int64_t K, int terms);
hipError_t launch_dense_product(const DenseProduct &c, char *ws, hipStream_t s);
//   Gradients in `dtype` from dy (B x M) and dense w (M x ldn), x (B x ldn) in the workspace;
//   fp16 products are multiplied by 2^*w_exponent (dx) and 2^*x_exponent (dw).  The first launch
//   leaves dbias as the layout's slabs of partial sums (rows of M), the second takes the products.
struct DenseGradLayout {
    size_t grad, part, sums, bytes;
    int64_t ldn, ldm, slabs;
};
struct DenseGrad {
    int dtype;
    const void *dy;
    int64_t B, lddy, M, N;
    const void *w, *x;
    const int *w_exponent, *x_exponent;
    void *dx;
    int64_t lddx;
    void *dw;
    int64_t lddw;
    float *dbias;
};
DenseGradLayout dense_grad_layout(size_t size, int64_t B, int64_t M, int64_t N, bool dx, bool dw,
                                  bool dbias);
hipError_t launch_dense_slabs(const DenseGrad &c, char *ws, hipStream_t s);
hipError_t launch_dense_grad(const DenseGrad &c, char *ws, hipStream_t s);

// Microscaled matrices (codes, their leading dimension in bytes, scale bytes without gaps).
struct MxMatrix {
    const uint8_t *codes;
    int64_t ld;
    const uint8_t *scale;
    int format;
};
// Codes and scale bytes, and, where values is not NULL, the bf16 numbers they stand for (up to
// whole groups); codes and scale may be NULL.  Unpack also writes zeros to columns cols ..
// padded - 1.
// order: codes and scale bytes in the order in which the few-rows product reads them (whole tiles
// of 16 rows, of which those past `rows` are left as they were, and whole pairs of 128 columns).
struct MxOrder {
    uint8_t *codes, *scale;
    int nbt;            // tiles of 16 rows
};
hipError_t launch_mx_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                          int format, uint8_t *codes, int64_t ldq, uint8_t *scale,
                          uint16_t *values, int64_t ldv, const MxOrder *order, hipStream_t s);
constexpr int kMxTops = 16;
struct MxShift {
    const int *tops;   // kMxTops scale bytes, the largest among them
    int *down;
};
hipError_t launch_mx_unpack(const MxMatrix &m, int64_t rows, int64_t cols, int dtype, void *out,
                            int64_t ldo, int64_t padded, hipStream_t s);
// The microscaled linear layer and its gradients.
struct MxLinearCall {
    MxMatrix w;
    int64_t M, N;
    const void *x;           // dense, of type dtype, or NULL: xq is given
    int64_t ldx;
    MxMatrix xq;
    bool keep;               // x is given and its codes are wanted in xq
    int dtype;
    int64_t B;
    const float *bias;
    const void *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
};
struct MxLayout {
    size_t codes, scale, xs, wvals, xvals, parts, bytes;
    int64_t ldq;             // of the codes in the workspace
    int64_t ldn;             // of unpacked rows
};
MxLayout mx_linear_layout(int format, int64_t B, int64_t M, int64_t N);
hipError_t launch_mx_linear(const MxLinearCall &c, char *ws, hipStream_t s);
struct MxGrad {
    int dtype;
    const void *dy;
    int64_t B, lddy, M, N;
    MxMatrix w, x;
    void *dx;
    int64_t lddx;
    void *dw;
    int64_t lddw;
    float *dbias;
};
size_t mx_grad_bytes(int dtype, int64_t B, int64_t M, int64_t N, bool dx, bool dw, bool dbias);
hipError_t launch_mx_grad(const MxGrad &c, char *ws, hipStream_t s);

// The paged cache of keys and values, and attention over it.
struct CacheShape {
    uint8_t *k_codes, *k_scale, *v_codes, *v_scale;
    int64_t pages;
    int heads, page_log2, dim, format;
};
struct CacheBatch {
    const int32_t *table;   // seqs x width page numbers, rows of ldt
    int64_t ldt, width;
    const int32_t *lens, *starts;
    int64_t seqs;
};
struct CacheRows {
    const void *p;          // rows x heads x dim values
    int64_t row, head;      // strides in values
};
hipError_t launch_cache_move(bool write, const CacheShape &c, const CacheBatch &b, int dtype,
                             const CacheRows &k, const CacheRows &v, int64_t rows, hipStream_t s);
struct AttentionCall {
    CacheShape c;
    CacheBatch b;
    int dtype;
    CacheRows q, o;         // rows x (heads x group) x dim
    int group;
    int64_t rows;
    float scale;
};
// Of this batch, and the most of it and every smaller one.
size_t attention_bytes(int dim, int group, int64_t seqs, int64_t rows);
size_t attention_most_bytes(int dim, int group, int64_t seqs, int64_t rows);
// Threads of the launch of large tiles (0: there is none), at most.
int64_t attention_threads(int group, int heads, int64_t seqs, int64_t rows);
hipError_t launch_attention(const AttentionCall &c, char *ws, hipStream_t s);

// 8-bit checkpoints (unpack also writes zeros to columns cols .. padded - 1 of out).
hipError_t launch_act_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int8_t *codes, int64_t ldq, uint8_t *scale, hipStream_t s);
hipError_t launch_act_unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale,
                             int64_t rows, int64_t cols, int dtype, void *out, int64_t ldo,
                             int64_t padded, hipStream_t s);

// Error feedback over coding blocks.
hipError_t launch_ldlq_update(float *tgt, int64_t ldt, const float *W, int64_t ldw,
                              const float *what, int64_t ldh, const float *U, int64_t ldu,
                              int64_t M, int64_t c_begin, int64_t c_end, int64_t i0, int T,
                              hipStream_t s);
hipError_t launch_ldlq_scatter(const uint32_t *sbits, const uint32_t *sstart,
                               const float *scost, int64_t M, int nwords, int64_t nbpr,
                               int64_t j, uint32_t *bitstream, uint32_t *start_state,
                               float *cost, hipStream_t s);

// L = 16 register-resident path.
bool l16_supported(const Problem &p);
size_t l16_fixed_bytes(const Problem &p);
size_t l16_bp_bytes(const Problem &p);
hipError_t launch_l16_prepare(const Problem &p, const float *C, char *fixed_ws, hipStream_t s);
hipError_t launch_acs_l16(const Problem &p, const Plan &pl, const float *W, const float *d,
                          int64_t block0, int64_t nb, char *ws, float *cost, hipStream_t s);
// swap_halves: the k*V = 4 kernel's relabelled trellis (kernels_l16h.hip)
hipError_t launch_traceback_l16(const Problem &p, const Plan &pl, int64_t block0, int64_t nb,
                                const char *ws, uint32_t *bitstream, uint32_t *start_state,
                                hipStream_t s, bool swap_halves = false);

// L = 16, k*V = 4 register-resident path (half-steps).
bool l16h_supported(const Problem &p);
size_t l16h_fixed_bytes(const Problem &p);
size_t l16h_bp_bytes(const Problem &p);
hipError_t launch_l16h_prepare(const Problem &p, const float *C, char *fixed_ws, hipStream_t s);
hipError_t launch_acs_l16h(const Problem &p, const Plan &pl, const float *W, const float *d,
                           int64_t block0, int64_t nb, char *ws, float *cost, hipStream_t s);

// L = 16, k*V = 3 register-resident path.
bool l16k3_supported(const Problem &p);
size_t l16k3_fixed_bytes(const Problem &p);
size_t l16k3_bp_bytes(const Problem &p);
hipError_t launch_l16k3_prepare(const Problem &p, const float *C, char *fixed_ws,
                                hipStream_t s);
hipError_t launch_acs_l16k3(const Problem &p, const Plan &pl, const float *W, const float *d,
                            int64_t block0, int64_t nb, char *ws, float *cost, hipStream_t s);
hipError_t launch_traceback_l16k3(const Problem &p, const Plan &pl, int64_t block0, int64_t nb,
                                  const char *ws, uint32_t *bitstream, uint32_t *start_state,
                                  hipStream_t s);

// Workspace layout helpers: [fixed area][per-block area x batch]
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace tcq
