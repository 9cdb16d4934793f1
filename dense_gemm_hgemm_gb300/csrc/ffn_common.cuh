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

// ---- results anywhere, of rows on the boundaries: neighbouring lanes hold neighbouring packs of W words, and a lane
// stores what lies between two boundaries, the end of the lane's pack before it and the start of its own.  The first
// lane of a warp or row and the last one store the rest of theirs element by element.  (All lanes of a warp come here.)
//   p: where the pack goes, n: elements of the row from there on (none: <= 0), lanes: of the row
template <typename E, int W>
__device__ __forceinline__ void store_between(const uint32_t (&w)[W], E* p, int n, int lanes) {
    constexpr int kUnit = W * 4 < 16 ? W * 4 : 16, kEach = W * 4 / 8;       // bytes between boundaries, of an element
    constexpr int kBefore = kUnit / 4;                                      // words of the lane before that may be needed
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (kUnit - 1)), words = off / 4, bits = off % 4 * 8;
    const int lane = static_cast<int>(threadIdx.x) & (lanes < 32 ? lanes - 1 : 31);
    uint32_t v[kBefore + W];
#pragma unroll
    for (int i = 0; i < kBefore; ++i) v[i] = __shfl_up_sync(0xffffffffu, w[W - kBefore + i], 1);
#pragma unroll
    for (int i = 0; i < W; ++i) v[kBefore + i] = w[i];
    if (n <= 0) return;
    const bool first = lane == 0, last = lane == (lanes < 32 ? lanes - 1 : 31) || n <= 8;
    const int here = W * 4 - off;                                           // bytes of the own pack's part
    if (!first) {
        // v moved up by off bytes
        if constexpr (kEach < 4) {
#pragma unroll
            for (int i = kBefore + W - 1; i > 0; --i) v[i] = __funnelshift_l(v[i - 1], v[i], bits);
        }
#pragma unroll
        for (int i = kBefore + W - 1; i > 0; --i) v[i] = words & 1 ? v[i - 1] : v[i];
        char* to = reinterpret_cast<char*>(p) - off;
        if constexpr (kUnit == 16) {
#pragma unroll
            for (int i = kBefore + W - 1; i > 1; --i) v[i] = words & 2 ? v[i - 2] : v[i];
#pragma unroll
            for (int i = 0; i < W; i += 4)
                *reinterpret_cast<uint4*>(to + i * 4) = make_uint4(v[kBefore + i], v[kBefore + i + 1], v[kBefore + i + 2], v[kBefore + i + 3]);
        } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(v[kBefore], v[kBefore + 1]);
        }
    }
    if (first || last) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * kEach < here ? first : last) p[i] = static_cast<E>(w[i * kEach / 4] >> (i * kEach % 4 * 8));
    }
}
// An Eight or eight bytes of a result, placed as its columns (OFF: anywhere, see above).
template <bool WHOLE, bool OFF, typename T>
__device__ __forceinline__ void store_result(const Eight<T>& v, T* p, int n, int lanes) {
    if constexpr (OFF) {
        constexpr int kWords = 4 * Eight<T>::kParts;
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(&v.part[i / 4].raw)[i % 4];
        store_between(w, reinterpret_cast<typename RawOf<static_cast<int>(sizeof(T))>::type*>(p), n, lanes);
    } else {
        v.template store<WHOLE>(p, n);
    }
}
template <bool WHOLE, bool OFF>
__device__ __forceinline__ void store_result(uint2 v, uint8_t* p, int n, int lanes) {
    if constexpr (OFF) {
        const uint32_t w[2] = {v.x, v.y};
        store_between(w, p, n, lanes);
    } else {
        store_bytes<WHOLE>(p, n, v);
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
