// Decoding of eight consecutive weights at a time (device code shared by the coded linear
// layer's kernels).
//
// A chunk is 8 columns of one coding block, 8 / V steps.  Its states are L-bit windows
// (L <= 16) of s_0 || b_1 || ... that end at most 8 k bits apart, so they lie in the
// 8 k + 16 - kV bits before the chunk's end: NW words, shifted once so that the chunk's last
// bit is bit 0.  Each state then is one bit-field extract with constant offsets.  A chunk's
// outputs are 16 bytes of a 16-bit type, so neighbouring lanes store neighbouring pieces.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tcq {

template <int KV, int V>
struct Chunk {
    static_assert(8 % V == 0 && KV % V == 0, "whole steps per chunk");
    static constexpr int kSteps = 8 / V;
    static constexpr int kBits = 8 * KV / V;           // fresh bits of a chunk
    static constexpr int NW = (kBits + 16 - KV + 31) / 32;
};

// The words of chunk q of the block whose stream is wb and start state s0, with the
// chunk's last bit at bit 0 of n[0].
template <int KV, int V>
__device__ __forceinline__ void chunk_words(const uint32_t *wb, const uint32_t *s0, int q,
                                            uint32_t (&w)[Chunk<KV, V>::NW + 1]) {
    using C = Chunk<KV, V>;
    const int j = ((q + 1) * C::kBits - 1) >> 5;  // word of the chunk's last bit
#pragma unroll
    for (int i = 0; i <= C::NW; ++i) {
        // (words before s_0 are past every window: any value does)
        const uint32_t *p = j - i >= 0 ? wb + (j - i) : s0;
        w[i] = *p;
    }
}

template <int KV, int V>
__device__ __forceinline__ void chunk_align(const uint32_t (&w)[Chunk<KV, V>::NW + 1], int q,
                                            uint32_t (&n)[Chunk<KV, V>::NW]) {
    using C = Chunk<KV, V>;
    const int e = (q + 1) * C::kBits;
    const int sh = (32 - (e & 31)) & 31;
#pragma unroll
    for (int i = 0; i < C::NW; ++i) n[i] = __builtin_amdgcn_alignbit(w[i + 1], w[i], sh);
}

// State of step t (a constant once unrolled).
template <int KV, int V>
__device__ __forceinline__ uint32_t chunk_state(const uint32_t (&n)[Chunk<KV, V>::NW], int t,
                                                int L) {
    using C = Chunk<KV, V>;
    const int off = (C::kSteps - 1 - t) * KV;
    const int i = off / 32;
    if (off % 32 + 16 <= 32 || i + 1 >= C::NW)
        return __builtin_amdgcn_ubfe(n[i], off % 32, L);
    return __builtin_amdgcn_ubfe(__builtin_amdgcn_alignbit(n[i + 1], n[i], off % 32), 0, L);
}

// Four chunks of one run of 32 columns (K = kV / V words, word-aligned) from the run's words
// w[1 .. K] and the word before them, w[0]: every shift is a constant.
template <int KV, int V>
__device__ __forceinline__ void run_align(const uint32_t (&w)[KV / V + 1], int s,
                                          uint32_t (&n)[Chunk<KV, V>::NW]) {
    using C = Chunk<KV, V>;
    const int e = (s + 1) * C::kBits;
    const int j = (e - 1) / 32, sh = (32 - e % 32) % 32;
#pragma unroll
    for (int i = 0; i < C::NW; ++i) {
        // (words before w[0] are past every window)
        const uint32_t lo = j - i >= -1 ? w[j - i + 1] : 0u;
        const uint32_t hi = j - i - 1 >= -1 ? w[j - i] : 0u;
        n[i] = sh ? __builtin_amdgcn_alignbit(hi, lo, sh) : lo;
    }
}

// Registers r[s] of lane group g (16 lanes each) to registers r[g] of lane group s.
__device__ __forceinline__ void transpose4(uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                           uint32_t &r3) {
    auto a = __builtin_amdgcn_permlane32_swap(r0, r2, false, false);
    auto b = __builtin_amdgcn_permlane32_swap(r1, r3, false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    r0 = c[0];
    r1 = c[1];
    r2 = d[0];
    r3 = d[1];
}

// `bytes` (a multiple of 16) of a table part from global memory straight into LDS, by THREADS
// threads; the caller waits (vmcnt 0) and meets the workgroup afterwards.  `vec`: src is
// 16-byte aligned; else the values (size 2 or 4) are copied one by one.
template <int THREADS>
__device__ __forceinline__ void table_to_lds(char *lds, const char *src, int bytes, int size,
                                             bool vec, int tid) {
    if (vec) {
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(src), 0, bytes, 0x00020000);
        const int wave0 = __builtin_amdgcn_readfirstlane(tid & ~63);
        for (int at = 0; at < bytes; at += THREADS * 16) {
            // (whole waves past the end are skipped; lanes past it load zeros, inside the
            // 1 KiB that the caller leaves for a part smaller than that)
            if (at + wave0 * 16 < bytes)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rs, (__attribute__((address_space(3))) void *)(lds + at + wave0 * 16), 16,
                    at + tid * 16, 0, 0, 0);
        }
    } else if (size == 2) {
        for (int i = tid; i < bytes / 2; i += THREADS)
            reinterpret_cast<uint16_t *>(lds)[i] = reinterpret_cast<const uint16_t *>(src)[i];
    } else {
        for (int i = tid; i < bytes / 4; i += THREADS)
            reinterpret_cast<uint32_t *>(lds)[i] = reinterpret_cast<const uint32_t *>(src)[i];
    }
}

}  // namespace tcq
