// ffn_quant.cu -- conversion of a matrix to e4m3 with scales (gemm_ffn.h).
#include <type_traits>

#include "ffn_common.cuh"

namespace gbt {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kSide = 128;                   // a block's tile: 128 x 128 elements
// Eights that a thread holds: of 128 rows, or of 64 where nothing joins a tile's rows (more blocks
// an SM: 8192 x 8192 bf16 45 -> 39 us).  Element by element 16-bit types spill 20 to 40 bytes a thread at these caps.
template <bool SQUARE, bool TRANSPOSE>
constexpr int kHeld = SQUARE || TRANSPOSE ? 8 : 4;

struct QuantArgs {
    const void* x;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldq, lds;
    int rows, cols, tiles_across;
};

// A block converts one tile of 128 x 128 elements, which its threads keep in registers between
// the largest value and the conversion: x is read once and q written once, 32 KB of bf16 in
// flight a block.  16 threads hold a row's 128 columns (as Eight has them), each of eight rows:
// t / 16 + 16 k, or, transposed, 8 (t / 16) + k, so that a column's eight values are eight
// bytes of a result's row.  That goes through shared memory, its 8-byte units exchanged
// within a row by `turn` so that no two lanes of a store or a load meet in a bank.
// WHOLE: of x and of q (see Eight).  (Rows and columns of a tile behind 2^31 - 1 elements stay below 2^31: tiles
// divide it.)
template <typename T, bool SQUARE, bool TRANSPOSE, bool WHOLE>
__global__ void __launch_bounds__(kQuantThreads, (sizeof(T) == 2 ? 3 : 2) + (kHeld<SQUARE, TRANSPOSE> == 4 ? 2 : 0))
    quantize_kernel(const QuantArgs a) {
    constexpr int kPacks = kHeld<SQUARE, TRANSPOSE>;
    __shared__ uint32_t high[kSide];                             // sizes, as bits (their order is the numbers')
    __shared__ alignas(16) uint2 turned[TRANSPOSE ? kSide * kSide / 8 : 1];
    const int tid = static_cast<int>(threadIdx.x), at = tid % 16, row = tid / 16;
    const int row0 = static_cast<int>(blockIdx.x / a.tiles_across) * (16 * kPacks);
    const int col0 = static_cast<int>(blockIdx.x % a.tiles_across) * kSide;
    const int c = col0 + first_column<WHOLE>(at), left = a.cols - c;
    const auto column = [&](int i) { return WHOLE ? at * 8 + i : at + kApart * i; };    // of the tile
    const auto turn = [](int col) { return WHOLE ? col / 8 : col % 16; };
    if (tid < kSide) high[tid] = 0;
    wait_for_previous_kernel();
    let_next_kernel_start();
    Eight<T> held[kPacks];
#pragma unroll
    for (int k = 0; k < kPacks; ++k) {
        const int r = row0 + (TRANSPOSE ? row * 8 + k : row + 16 * k);
        held[k].template load<WHOLE>(static_cast<const T*>(a.x) + r * a.ldx + c, r < a.rows ? left : 0);
    }
    if constexpr (SQUARE || TRANSPOSE) __syncthreads();
    if constexpr (SQUARE) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < kPacks; ++k) {
            Pair v[4];
            held[k].get(v);
            m = fmaxf(m, largest(v));
        }
        m = warp_max(m);
        if (tid % 32 == 0) atomicMax(&high[0], __float_as_uint(m));
        __syncthreads();
    } else if constexpr (TRANSPOSE) {
        // the largest of each column: over a thread's rows, the warp's two, and the warps
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < kPacks; ++k) m = fmaxf(m, fabsf(held[k].get(i)));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            if (tid % 32 < 16) atomicMax(&high[column(i)], __float_as_uint(m));
        }
        __syncthreads();
    }
    if constexpr (!TRANSPOSE) {
        float square = 0.f, inverse = 0.f;
        if constexpr (SQUARE) {
            square = scale_of(__uint_as_float(high[0]));
            inverse = 1.f / square;
            if (tid == 0) a.scales[row0 / kSide * a.lds + col0 / kSide] = square;
        }
#pragma unroll
        for (int k = 0; k < kPacks; ++k) {
            const int r = row0 + row + 16 * k;
            Pair v[4];
            held[k].get(v);
            if constexpr (!SQUARE) {
                const float s = scale_of(largest_of_group(largest(v)));
                inverse = 1.f / s;
                if (at == 0 && r < a.rows) a.scales[r * a.lds + col0 / kSide] = s;
            }
            store_bytes<WHOLE>(a.q + r * a.ldq + c, r < a.rows ? left : 0, e4m3_eight(v, inverse));
        }
    } else {
        // q's row is x's column: its scale index runs along x's rows
        if constexpr (SQUARE) {
            if (tid == 0) a.scales[col0 / kSide * a.lds + row0 / kSide] = scale_of(__uint_as_float(high[0]));
        } else {
            if (tid < kSide && col0 + tid < a.cols)
                a.scales[(col0 + tid) * a.lds + row0 / kSide] = scale_of(__uint_as_float(high[tid]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float inverse = 1.f / scale_of(__uint_as_float(high[SQUARE ? 0 : column(i)]));
            Pair down[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) down[k] = Pair(held[2 * k].get(i), held[2 * k + 1].get(i));
            turned[column(i) * 16 + (row ^ turn(column(i)))] = e4m3_eight(down, inverse);
        }
        __syncthreads();
        // 128 rows of 128 bytes, eight a thread and step
#pragma unroll
        for (int k = 0; k < kSide / 16; ++k) {
            const int r = row + 16 * k, n = col0 + r < a.cols ? a.rows - row0 - column(0) : 0;
            uint8_t* to = a.q + (col0 + r) * a.ldq + row0 + column(0);
            if constexpr (WHOLE) {
                store_bytes<true>(to, n, turned[r * 16 + (at ^ turn(r))]);
            } else {
                const uint8_t* bytes = reinterpret_cast<const uint8_t*>(turned + r * 16);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int b = column(i);
                    if (kApart * i < n) to[kApart * i] = bytes[((b / 8) ^ turn(r)) * 8 + b % 8];
                }
            }
        }
    }
}

}  // namespace
}  // namespace gbt

extern "C" gemm_status_t gemm_fp8_quantize(int64_t rows, int64_t cols, gemm_elem_t elem, const void* x,
                                           int64_t ldx, gemm_scale_t kind, int32_t transpose, void* q,
                                           int64_t ldq, float* scales, int64_t lds, void* stream) {
    using namespace gbt;
    if (!valid_elem(elem) || (kind != GEMM_SCALE_ROW && kind != GEMM_SCALE_SQUARE)) return GEMM_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX || (transpose != 0 && transpose != 1))
        return GEMM_ERR_INVALID_ARG;
    const int64_t down = groups_of(rows), across = groups_of(cols);
    if (down * across > (int64_t{1} << 29)) return GEMM_ERR_INVALID_ARG;
    const int64_t out_cols = transpose ? rows : cols;
    if (rows > 0 && cols > 0 && (!x || !q || !scales || ldx < cols || ldq < out_cols || lds < groups_of(out_cols)))
        return GEMM_ERR_INVALID_ARG;
    const int e = elem_bytes(elem);
    if (!aligned(x, e) || !aligned(scales, 4)) return GEMM_ERR_ALIGNMENT;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (rows == 0 || cols == 0) return GEMM_OK;
    const QuantArgs a{x, static_cast<uint8_t*>(q), scales, ldx, ldq, lds, static_cast<int>(rows), static_cast<int>(cols),
                      static_cast<int>(across)};
    const bool whole = cols % 8 == 0 && out_cols % 8 == 0 && rows_aligned(x, ldx, e) && bytes_aligned(q, ldq);
    const Queue queue{stream, device};
    return with_elem(elem, [&](auto t) {
        using T = decltype(t);
        const auto go = [&](auto square, auto turned) {
            constexpr bool kSquare = decltype(square)::value, kTurned = decltype(turned)::value;
            constexpr int kRows = 16 * kHeld<kSquare, kTurned>;
            const int64_t tiles = (rows + kRows - 1) / kRows * across;
            return whole ? launch<quantize_kernel<T, kSquare, kTurned, true>>(tiles, kQuantThreads, 0, queue, 1, a)
                         : launch<quantize_kernel<T, kSquare, kTurned, false>>(tiles, kQuantThreads, 0, queue, 1, a);
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (kind == GEMM_SCALE_ROW) return transpose ? go(No(), Yes()) : go(No(), No());
        return transpose ? go(Yes(), Yes()) : go(Yes(), No());
    });
}
