// ffn_common.cuh -- what the kernels of gemm_ffn.h share: groups of eight columns of any
// type and alignment, and e4m3 numbers with their scales.
#pragma once
#include "gemm_ffn.h"
#include "train_common.cuh"

namespace gbt {

constexpr int kGroup = 128;                    // elements that share a scale
constexpr float kE4m3Top = 448.f;              // the largest e4m3 number
constexpr float kLeastScale = 1.17549435e-38f; // 2^-126: one over it is a normal number

inline int64_t groups_of(int64_t cols) { return (cols + kGroup - 1) / kGroup; }

// Eight columns of a row as they are in memory, of the 128 that 16 threads hold together.
// WHOLE: rows start at 16-byte boundaries and have a multiple of eight columns; a thread has
// eight neighbours, which move together or not at all (no branch: all loads of a thread are in
// flight at once).  Else it has every 16th, element by element: the 16 threads' accesses are
// neighbours (neighbours of a thread made each access 32 sectors of a warp).
constexpr int kApart = 16;
template <bool WHOLE>
__device__ __forceinline__ int first_column(int thread) {
    return WHOLE ? thread * 8 : (thread & ~15) * 8 + (thread & 15);
}
template <typename T>
struct Eight {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T)), kParts = 8 / kPer;
    Pack<T, kPer> part[kParts];
    template <bool WHOLE>
    __device__ __forceinline__ void load(const T* p, int n) {
        if constexpr (WHOLE) {
#pragma unroll
            for (int k = 0; k < kParts; ++k) {
                part[k].clear();
                if (n > 0) part[k].raw = *reinterpret_cast<const uint4*>(p + k * kPer);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i / kPer].set_raw(i % kPer, i * kApart < n ? p[i * kApart] : from_f32<T>(0.f));
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void store(T* p, int n) const {
        if constexpr (WHOLE) {
#pragma unroll
            for (int k = 0; k < kParts; ++k)
                if (n > 0) *reinterpret_cast<uint4*>(p + k * kPer) = part[k].raw;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i * kApart < n) p[i * kApart] = reinterpret_cast<const T*>(&part[i / kPer].raw)[i % kPer];
        }
    }
    __device__ __forceinline__ float get(int i) const { return part[i / kPer].get(i % kPer); }
    // ... and all of them in pairs, as fp32 instructions take them
    __device__ __forceinline__ void get(Pair (&v)[4]) const { to_pairs(part, v); }
    __device__ __forceinline__ void set(const Pair (&v)[4]) { from_pairs(v, part); }
};

// Two numbers as e4m3 (to nearest even, at most 448 in size): lo in the lower byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint2 e4m3_eight(const Pair (&v)[4], float inverse) {
    const Pair by(inverse, inverse);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        mul2(v[i], by).get(lo, hi);
        w[i] = e4m3_pair(lo, hi);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Eight bytes, placed as the columns of an Eight (WHOLE: p aligned to 8 bytes).
template <bool WHOLE>
__device__ __forceinline__ void store_bytes(uint8_t* p, int n, uint2 v) {
    if constexpr (WHOLE) {
        if (n > 0) *reinterpret_cast<uint2*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * kApart < n) p[i * kApart] = static_cast<uint8_t>((i < 4 ? v.x : v.y) >> (i % 4 * 8));
    }
}

// The largest size among eight numbers (NaN aside, which fmaxf passes over).
__device__ __forceinline__ float largest(const Pair (&v)[4]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        v[i].get(lo, hi);
        m = fmaxf(fmaxf(m, fabsf(lo)), fabsf(hi));
    }
    return m;
}
// ... among 16 lanes, which hold 128 columns, in each of them.
__device__ __forceinline__ float largest_of_group(float m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

__device__ __forceinline__ float scale_of(float largest) { return fmaxf(largest * (1.f / kE4m3Top), kLeastScale); }

// Whether rows of eight-element packs can move whole.
inline bool packs_aligned(const void* p, int64_t ld, int bytes) { return !p || rows_aligned(p, ld, bytes); }
inline bool bytes_aligned(const void* p, int64_t ld) { return aligned(p, 8) && ld % 8 == 0; }

}  // namespace gbt
