// ffn_rms.cu -- root-mean-square norm with the residual's addition (gemm_ffn.h).
#include <algorithm>
#include <new>
#include <type_traits>

#include "ffn_common.cuh"

struct gemm_rms_plan {
    int64_t max_rows, cols;
    gemm_elem_t elem, weight_elem;
    int device, num_sms;
    float* partial;      // [blocks][cols] sums of the weight's gradient
};

namespace gbt {
namespace {

constexpr int kRowPacks = 2;                  // packs of eight columns that a lane holds
constexpr int kLaneColumns = 8 * kRowPacks;
constexpr int kMostRowLanes = 1024;
constexpr int kRowColumns = kMostRowLanes * kLaneColumns;   // the longest row that a block holds

// Lanes that hold a row: up to 128 a power of two, so that a group divides a block of 128; 16 at least, which
// are the 128 columns of a scale.  More are a block of their own, whole warps (in powers of two, 8192 x 5120
// bf16 took 65 us instead of 52, to 8 bits 75 instead of 49, its gradient 77 instead of 66).
constexpr int kSharedBlock = 128;
int row_lanes(int64_t cols) {
    int lanes = 16;
    while (lanes < kSharedBlock && lanes * kLaneColumns < cols) lanes *= 2;
    if (lanes * kLaneColumns >= cols) return lanes;
    return static_cast<int>(std::min<int64_t>((cols + 32 * kLaneColumns - 1) / (32 * kLaneColumns) * 32, kMostRowLanes));
}
constexpr int row_block(int lanes) { return lanes < kSharedBlock ? kSharedBlock : lanes; }
// The block sizes that kernels are made for, each for lanes up to it.
template <typename F>
gemm_status_t with_block(int lanes, F f) {
    if (lanes <= kSharedBlock) return f(std::integral_constant<int, kSharedBlock>());
    if (lanes <= 256) return f(std::integral_constant<int, 256>());
    if (lanes <= 384) return f(std::integral_constant<int, 384>());
    if (lanes <= 512) return f(std::integral_constant<int, 512>());
    if (lanes <= 768) return f(std::integral_constant<int, 768>());
    return f(std::integral_constant<int, kMostRowLanes>());
}
// ... and those of the kernels whose results lie off the boundaries, fewer as they are rare (those of 1024 threads
// spill 8 bytes).
template <typename F>
gemm_status_t with_block_off(int lanes, F f) {
    if (lanes <= kSharedBlock) return f(std::integral_constant<int, kSharedBlock>());
    if (lanes <= 512) return f(std::integral_constant<int, 512>());
    return f(std::integral_constant<int, kMostRowLanes>());
}
// A thread's place in such a block.
template <int BLOCK>
struct RowPlace {
    int lane, group, groups, threads;
    __device__ __forceinline__ explicit RowPlace(int lanes) {
        const int tid = static_cast<int>(threadIdx.x);
        lane = BLOCK == kSharedBlock ? tid & (lanes - 1) : tid;
        group = BLOCK == kSharedBlock ? tid / lanes : 0;
        groups = BLOCK == kSharedBlock ? BLOCK / lanes : 1;
        threads = BLOCK == kSharedBlock ? BLOCK : lanes;
    }
};

// The sum over a row's lanes, in each of them.  part: one float per warp of the block (all of
// its threads meet here where a row has more than a warp).
template <int BLOCK>
__device__ __forceinline__ float row_sum(float v, int lanes, float* part) {
    if (lanes == 16) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    v = warp_sum(v);
    if (lanes == 32) return v;
    const int warp = static_cast<int>(threadIdx.x) / 32, warps = lanes / 32;
    if (threadIdx.x % 32 == 0) part[warp] = v;
    __syncthreads();
    const int l = static_cast<int>(threadIdx.x) % 32, first = lanes > kSharedBlock ? 0 : warp & -warps;
    return warp_sum(l < warps ? part[first + l] : 0.f);
}

template <typename T, typename W>
struct RmsForwardArgs {
    const T* x;
    const T* residual;
    const W* gamma;
    T* total;
    T* y;
    uint8_t* q;
    float* scales;
    float* rstd;
    int64_t ldx, ldr, ldt, ldy, ldq, lds, rows;
    float eps;
    int cols, lanes;
    bool total_along, y_along;   // at x's distance from the 16-byte boundaries
};

// x + residual as it is kept: an fp32 sum (one rounding), rounded to T.
template <typename T>
__device__ __forceinline__ void add_eight(Eight<T>& x, const Eight<T>& residual) {
    Pair v[4], r[4];
    x.get(v);
    residual.get(r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], r[i]);
    x.set(v);
}

// sum + the squares of eight columns
template <typename T>
__device__ __forceinline__ Pair add_squares(const Eight<T>& t, Pair sum) {
    Pair v[4];
    t.get(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fma2(v[i], v[i], sum);
    return sum;
}

__device__ __forceinline__ float both(Pair v) {
    float lo, hi;
    v.get(lo, hi);
    return lo + hi;
}

// y of eight columns from t, and its conversion where Q8 (all lanes of a warp come here).
template <typename T, typename W, bool Q8, bool WHOLE, bool OFF>
__device__ __forceinline__ void finish_eight(const RmsForwardArgs<T, W>& a, int64_t row, int c, int n, float rstd,
                                             const Eight<T>& t, const Eight<W>& gamma) {
    Pair y[4], w[4];
    t.get(y);
    gamma.get(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], Pair(rstd, rstd));
    if (a.gamma) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], w[i]);
    }
    if constexpr (Q8) {
        const float s = scale_of(largest_of_group(largest(y)));
        if (n > 0 && c % kGroup == 0) a.scales[row * a.lds + c / kGroup] = s;
        store_result<WHOLE, OFF>(e4m3_eight(y, 1.f / s), a.q + row * a.ldq + c, n, a.lanes);
    } else {
        Eight<T> out;
        out.set(y);
        store_result<WHOLE, OFF>(out, a.y + row * a.ldy + c, n, a.lanes);
    }
}

// What a lane needs of a row, as it is in memory.
template <typename T, bool WHOLE>
struct RmsInput {
    Eight<T> x[kRowPacks], r[kRowPacks];
    template <bool ALONE, typename W>
    __device__ __forceinline__ void load(const RmsForwardArgs<T, W>& a, int64_t row, int lane) {
        const bool there = row < a.rows;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = first_column<WHOLE>(k * a.lanes + lane);
            x[k].template load<WHOLE>(a.x + row * a.ldx + c, there ? a.cols - c : 0);
            if (!ALONE) r[k].template load<WHOLE>(a.residual + row * a.ldr + c, there && a.residual ? a.cols - c : 0);
        }
    }
};

// Blocks of a forward kernel that an SM's registers hold (80 a thread at most, 128 for fp32 rows, 64 without
// a residual).  The aligned and the shifted kernels fit them; element by element addresses and masks do not: those
// kernels spill 32 to 64 bytes a thread, the gradient's 20 to 92.
constexpr int forward_blocks_an_sm(int block, int bytes, bool alone) {
    const int threads = bytes == 4 ? 512 : alone ? 1024 : 768;
    return block < threads ? threads / block : 1;
}
// Whether a lane's registers hold the next row, too.
template <int BLOCK, typename T>
constexpr bool kForwardAhead = BLOCK <= (sizeof(T) == 4 ? 512 : 768);

// A row is held by `lanes` threads, 16 columns each: it is read once, and its sum of squares
// and results come from registers.  A block goes over rows blockIdx.x, + gridDim.x, ... (BLOCK /
// lanes at a time); the next row's loads are in flight during the present one's sum (not with
// 1024 threads, whose registers do not hold two rows).  ALONE: no residual.  OFF: results need not be
// on the boundaries (with WHOLE, which the inputs decide, so that a row's sum has one order wherever results go).
template <typename T, typename W, int BLOCK, bool Q8, bool WHOLE, bool ALONE, bool OFF>
__global__ void __launch_bounds__(BLOCK, forward_blocks_an_sm(BLOCK, sizeof(T), ALONE)) rms_forward_kernel(const RmsForwardArgs<T, W> a) {
    constexpr bool kAhead = kForwardAhead<BLOCK, T>;
    __shared__ float part[2][BLOCK / 32];
    const RowPlace<BLOCK> at(a.lanes);
    const int lane = at.lane, group = at.group, groups = at.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    wait_for_previous_kernel();
    let_next_kernel_start();
    int turn = 0;
    RmsInput<T, WHOLE> next;
    if (kAhead) next.template load<ALONE>(a, static_cast<int64_t>(blockIdx.x) * groups + group, lane);
    Eight<W> gamma[kRowPacks];
#pragma unroll
    for (int k = 0; k < kRowPacks; ++k) {
        const int c = first_column<WHOLE>(k * a.lanes + lane);
        gamma[k].template load<WHOLE>(a.gamma + c, a.gamma ? a.cols - c : 0);
    }
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        const bool there = row < a.rows;
        RmsInput<T, WHOLE> now;
        if constexpr (kAhead) {
            now = next;
            next.template load<ALONE>(a, row + step, lane);
        } else {
            now.template load<ALONE>(a, row, lane);
        }
        Pair squares(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            if (!ALONE && a.residual) add_eight(now.x[k], now.r[k]);
            squares = add_squares(now.x[k], squares);
        }
        if (a.total) {
#pragma unroll
            for (int k = 0; k < kRowPacks; ++k) {
                const int c = first_column<WHOLE>(k * a.lanes + lane);
                store_result<WHOLE, OFF>(now.x[k], a.total + row * a.ldt + c, there ? a.cols - c : 0, a.lanes);
            }
        }
        const float sum = row_sum<BLOCK>(both(squares), a.lanes, part[turn]);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
        if (a.rstd && there && lane == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = first_column<WHOLE>(k * a.lanes + lane);
            finish_eight<T, W, Q8, WHOLE, OFF>(a, row, c, there ? a.cols - c : 0, rstd, now.x[k], gamma[k]);
        }
    }
}

// ---- rows off the 16-byte boundaries, all inputs' by the same distance (the type's rows of one length
// and padding).  A lane holds Eights that start at the boundaries: row `shift` elements behind one has
// column 8 e - shift + i in element i of Eight e, and the first and the last Eight reach beyond the row
// (16 bytes move where one of them is the row's; the others' values are dropped, and not written).  What
// belongs to a column (weights, their gradients) is in shared memory, with a column's place at
// (column % 8) * stride + column / 8 + 1: lanes are neighbours there whatever the shift.  Element by element,
// as rms_forward_kernel moves such rows, 10000 x 5003 bf16 took 149 us (here 99, 70 in blocks of whole
// warps) and its gradient 198 (here 121, 88).  It keeps the rows whose Eights, one more than their columns
// need, would take twice the lanes (32768 x 1024 bf16, rows of 1027: 65 us, here 79; the gradient 88, here 96),
// fp32 results (16384 x 4096, rows of 4099: 164 us, here 186) and results of 8 bits, whose scales' columns no
// longer are a lane's (through shared memory, 165 us to 146 at 10000 x 5003, but 93 to 119 at 8192 x 4099 fp32).

struct Columns {
    int stride;
    __device__ __forceinline__ explicit Columns(int lanes) : stride(2 * lanes + 2) {}
    __device__ __forceinline__ int size() const { return 8 * stride; }
    __device__ __forceinline__ int at(int column) const { return (column & 7) * stride + (column >> 3) + 1; }   // from -8
};
constexpr size_t columns_bytes(int lanes) { return 8 * (2 * static_cast<size_t>(lanes) + 2) * sizeof(float); }

template <typename T>
__device__ __forceinline__ int shift_of(const T* row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// An Eight at a boundary, of which elements first .. end - 1 are the row's.
template <typename T>
__device__ __forceinline__ void load_part(Eight<T>& v, const T* p, int end) {
#pragma unroll
    for (int k = 0; k < Eight<T>::kParts; ++k) {
        v.part[k].clear();
        if (end > k * Eight<T>::kPer) v.part[k].raw = *reinterpret_cast<const uint4*>(p + k * Eight<T>::kPer);
    }
}
template <typename T>
__device__ __forceinline__ void keep_part(Eight<T>& v, int first, int end) {
    if (first <= 0 && end >= 8) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < first || i >= end) v.part[i / Eight<T>::kPer].set_raw(i % Eight<T>::kPer, from_f32<T>(0.f));
}
// (along: p is at a boundary)
template <typename T>
__device__ __forceinline__ void store_part(const Eight<T>& v, T* p, int first, int end, bool along) {
    if (along && first <= 0 && end >= 8) {
        v.template store<true>(p, 8);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= first && i < end) p[i] = reinterpret_cast<const T*>(&v.part[i / Eight<T>::kPer].raw)[i % Eight<T>::kPer];
}

// The weights (ones where there are none) at their columns' places, zeros at the others; all loads of a
// thread are in flight at once.
template <typename W>
__device__ __forceinline__ void place_weights(float* room, const Columns& places, const W* gamma, int cols, int lanes, int threads) {
    constexpr int kEach = kLaneColumns + 1;          // of 16 columns a lane, and eight in front
    const int first = static_cast<int>(threadIdx.x) - 8;
    float v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int c = first + j * threads;
        v[j] = c < 0 || c >= cols ? 0.f : gamma ? to_f32(gamma[c]) : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int c = first + j * threads;
        if (c < lanes * kLaneColumns) room[places.at(c)] = v[j];
    }
}

template <typename T>
struct ShiftedInput {
    Eight<T> x[kRowPacks], r[kRowPacks];
    template <typename W>
    __device__ __forceinline__ void load(const RmsForwardArgs<T, W>& a, int64_t row, int lane) {
        const T* from = a.x + row * a.ldx;
        const int shift = shift_of(from);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift, end = row < a.rows ? a.cols - c : 0;
            load_part(x[k], from + c, end);
            load_part(r[k], a.residual + row * a.ldr + c, a.residual ? end : 0);
        }
    }
};

// As rms_forward_kernel, for results of T.
template <typename T, typename W, int BLOCK>
__global__ void __launch_bounds__(BLOCK, forward_blocks_an_sm(BLOCK, sizeof(T), false)) rms_forward_shifted_kernel(const RmsForwardArgs<T, W> a) {
    constexpr bool kAhead = kForwardAhead<BLOCK, T>;
    extern __shared__ float room[];              // the weights
    __shared__ float part[2][BLOCK / 32];
    const Columns places(a.lanes);
    const RowPlace<BLOCK> at(a.lanes);
    const int lane = at.lane, group = at.group, groups = at.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    wait_for_previous_kernel();
    let_next_kernel_start();
    ShiftedInput<T> next;
    if (kAhead) next.load(a, static_cast<int64_t>(blockIdx.x) * groups + group, lane);
    place_weights(room, places, a.gamma, a.cols, a.lanes, at.threads);
    __syncthreads();
    const float* const weights = room + lane;
    int turn = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        const bool there = row < a.rows;
        ShiftedInput<T> now;
        if constexpr (kAhead) {
            now = next;
            next.load(a, row + step, lane);
        } else {
            now.load(a, row, lane);
        }
        const int shift = shift_of(a.x + row * a.ldx);
        Pair squares(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift, end = there ? a.cols - c : 0;
            if (a.residual) add_eight(now.x[k], now.r[k]);
            keep_part(now.x[k], -c, end);
            squares = add_squares(now.x[k], squares);
            if (a.total) store_part(now.x[k], a.total + row * a.ldt + c, -c, end, a.total_along);
        }
        const float sum = row_sum<BLOCK>(both(squares), a.lanes, part[turn]);
        turn ^= 1;
        const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
        if (a.rstd && there && lane == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift;
            Pair y[4];
            now.x[k].get(y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Pair w(weights[places.at(2 * i - shift) + k * a.lanes], weights[places.at(2 * i + 1 - shift) + k * a.lanes]);
                y[i] = mul2(mul2(y[i], Pair(rstd, rstd)), w);
            }
            Eight<T> out;
            out.set(y);
            store_part(out, a.y + row * a.ldy + c, -c, there ? a.cols - c : 0, a.y_along);
        }
    }
}

// Longer rows: a block goes over its row twice.
template <typename T, typename W, bool Q8, bool WHOLE, bool OFF>
__global__ void __launch_bounds__(kMostRowLanes) rms_forward_wide_kernel(const RmsForwardArgs<T, W> a) {
    __shared__ float part[kMostRowLanes / 32];
    const int64_t row = blockIdx.x;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const T* x = a.x + row * a.ldx;
    const T* residual = a.residual ? a.residual + row * a.ldr : nullptr;
    T* total = a.total ? a.total + row * a.ldt : nullptr;
    const auto sum_at = [&](int c, int n, Eight<T>& t) {
        Eight<T> r;
        t.template load<WHOLE>(x + c, n);
        r.template load<WHOLE>(residual + c, residual ? n : 0);
        if (residual) add_eight(t, r);
    };
    Pair squares(0.f, 0.f);
    for (int c0 = 0; c0 < a.cols; c0 += kMostRowLanes * 8) {
        const int c = c0 + first_column<WHOLE>(static_cast<int>(threadIdx.x)), n = a.cols - c;
        if (!OFF && n <= 0) break;
        Eight<T> t;
        sum_at(c, n, t);
        squares = add_squares(t, squares);
        if (total) store_result<WHOLE, OFF>(t, total + c, n, kMostRowLanes);
    }
    const float sum = row_sum<kMostRowLanes>(both(squares), kMostRowLanes, part);
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // (a thread reads back only what it wrote: total may be x or the residual, and then lies where they do.  All
    // lanes of a warp go through every step: the largest value of a group is taken among them.)
    for (int c0 = 0; c0 < a.cols; c0 += kMostRowLanes * 8) {
        const int c = c0 + first_column<WHOLE>(static_cast<int>(threadIdx.x)), n = a.cols - c;
        Eight<T> t;
        Eight<W> gamma;
        gamma.template load<WHOLE>(a.gamma + c, a.gamma ? n : 0);
        if (total && (!OFF || a.total_along)) {
            t.template load<WHOLE>(total + c, n);
        } else {
            sum_at(c, n, t);
        }
        finish_eight<T, W, Q8, WHOLE, OFF>(a, row, c, n, rstd, t, gamma);
    }
}

// ---------------------------------------------------------------- backward

template <typename T, typename W>
struct RmsBackwardArgs {
    const T* total;
    const W* gamma;
    const float* rstd;
    const T* dy;
    const T* dtotal;
    T* dx;
    float* partial;             // [grid][cols], or NULL: no gradient of gamma wanted
    int64_t ldt, lddy, lddt, lddx, rows;
    int cols, lanes;
    bool dx_along;               // at total's distance from the 16-byte boundaries
};

// What a lane needs of a row, as it is in memory (MORE: dtotal too).
template <typename T, bool WHOLE, bool MORE>
struct RmsRow {
    Eight<T> t[kRowPacks], dy[kRowPacks], more[kRowPacks];
    float rstd;
    template <typename W>
    __device__ __forceinline__ void load(const RmsBackwardArgs<T, W>& a, int64_t row, int lane) {
        const bool there = row < a.rows;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = first_column<WHOLE>(k * a.lanes + lane), n = there ? a.cols - c : 0;
            t[k].template load<WHOLE>(a.total + row * a.ldt + c, n);
            dy[k].template load<WHOLE>(a.dy + row * a.lddy + c, n);
            if (MORE) more[k].template load<WHOLE>(a.dtotal + row * a.lddt + c, a.dtotal ? n : 0);
        }
        rstd = there ? a.rstd[row] : 0.f;
    }
};

// v * rstd + what reaches the sum on its other way, with one rounding: written as a product and a sum, the assembler
// made one operation of them in some kernels and not in others, and the same row had other bits in each.
__device__ __forceinline__ Pair along_total(Pair v, float rstd, Pair more, const void* dtotal) {
    return dtotal ? fma2(v, Pair(rstd, rstd), more) : mul2(v, Pair(rstd, rstd));
}

// Blocks of a backward kernel that share an SM (its registers: 128 a thread).
constexpr int backward_blocks_an_sm(int block) { return block < 512 ? 512 / block : 1; }
// Whether a lane's registers hold the next row, too ...
template <int BLOCK, typename T>
constexpr bool kBackwardAhead = BLOCK <= (sizeof(T) == 4 ? 512 : 768);
// ... and of that dtotal, too; and the weights and their gradient.
template <int BLOCK>
constexpr bool kBackwardMore = BLOCK <= 512;
template <int BLOCK, typename T>
constexpr bool kBackwardRoom = BLOCK <= 512 && sizeof(T) == 2;

// A block goes over rows blockIdx.x, + gridDim.x, ... (BLOCK / lanes at a time) and keeps its
// share of the weight's gradient in registers, 16 columns a lane.  The next row's loads are in
// flight during the present one's sum (not with 1024 threads, whose registers do not hold two rows;
// above 512 dtotal is loaded where it is used).  So are gamma, and the weight's gradient is in shared
// memory, above 512 threads and with fp32 rows, which take twice the registers.
template <typename T, typename W, int BLOCK, bool WHOLE, bool OFF>
__global__ void __launch_bounds__(BLOCK, backward_blocks_an_sm(BLOCK)) rms_backward_kernel(const RmsBackwardArgs<T, W> a) {
    constexpr bool kAhead = kBackwardAhead<BLOCK, T>, kMore = kBackwardMore<BLOCK>, kRoom = kBackwardRoom<BLOCK, T>;
    extern __shared__ Pair shared[];             // the weight's gradient: of each thread, or of several groups
    __shared__ float part[2][BLOCK / 32];
    const RowPlace<BLOCK> at(a.lanes);
    const int lane = at.lane, group = at.group, groups = at.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const auto kept = [&](int k, int i) -> Pair& { return shared[(k * 4 + i) * BLOCK + threadIdx.x]; };
    Pair dgamma[kRowPacks][4];
#pragma unroll
    for (int k = 0; k < kRowPacks; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) (kRoom ? dgamma[k][i] : kept(k, i)) = Pair(0.f, 0.f);
    }
    int turn = 0;
    Eight<W> gamma[kRowPacks];
    const auto load_gamma = [&](int k) {
        const int c = first_column<WHOLE>(k * a.lanes + lane);
        gamma[k].template load<WHOLE>(a.gamma + c, a.gamma ? a.cols - c : 0);
    };
    if constexpr (kRoom) {
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) load_gamma(k);
    }
    RmsRow<T, WHOLE, kMore> next;
    if (kAhead) next.load(a, static_cast<int64_t>(blockIdx.x) * groups + group, lane);
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        RmsRow<T, WHOLE, kMore> now;
        if constexpr (kAhead) {
            now = next;
            next.load(a, row + step, lane);
        } else {
            now.load(a, row, lane);
        }
        // (hat and g are made twice: kept over the sum, they would take the next row's registers)
        const auto hat_and_g = [&](int k, Pair (&hat)[4], Pair (&d)[4], Pair (&g)[4]) {
            if constexpr (!kRoom) load_gamma(k);
            now.t[k].get(hat);
            now.dy[k].get(d);
            gamma[k].get(g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hat[i] = mul2(hat[i], Pair(now.rstd, now.rstd));
                g[i] = a.gamma ? mul2(d[i], g[i]) : d[i];
            }
        };
        Pair products(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            Pair hat[4], d[4], g[4];
            hat_and_g(k, hat, d, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Pair& to = kRoom ? dgamma[k][i] : kept(k, i);
                to = fma2(d[i], hat[i], to);
                products = fma2(g[i], hat[i], products);
            }
        }
        if (!a.dx) continue;                     // (all of the block)
        const float mean = row_sum<BLOCK>(both(products), a.lanes, part[turn]) / static_cast<float>(a.cols);
        turn ^= 1;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = first_column<WHOLE>(k * a.lanes + lane), n = row < a.rows ? a.cols - c : 0;
            Pair hat[4], d[4], g[4];
            hat_and_g(k, hat, d, g);
            if constexpr (!kMore) now.more[k].template load<WHOLE>(a.dtotal + row * a.lddt + c, a.dtotal ? n : 0);
            now.more[k].get(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = along_total(fma2(hat[i], Pair(-mean, -mean), g[i]), now.rstd, d[i], a.dtotal);
            }
            Eight<T> out;
            out.set(g);
            store_result<WHOLE, OFF>(out, a.dx + row * a.lddx + c, n, a.lanes);
        }
    }
    if (!a.partial) return;
    if constexpr (!kRoom) {
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dgamma[k][i] = kept(k, i);
        }
    }
    float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    if (groups > 1) {
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kept(k, i) = dgamma[k][i];
        }
        __syncthreads();
        if (group != 0) return;
        for (int other = 1; other < groups; ++other) {
#pragma unroll
            for (int k = 0; k < kRowPacks; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dgamma[k][i] = add2(dgamma[k][i], shared[(k * 4 + i) * BLOCK + other * a.lanes + lane]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kRowPacks; ++k) {
        const int c = first_column<WHOLE>(k * a.lanes + lane);
        Eight<float> out;
        out.set(dgamma[k]);
        out.template store<WHOLE>(to + c, a.cols - c);
    }
}

template <typename T, bool MORE>
struct ShiftedRow {
    Eight<T> t[kRowPacks], dy[kRowPacks], more[kRowPacks];
    float rstd;
    template <typename W>
    __device__ __forceinline__ void load(const RmsBackwardArgs<T, W>& a, int64_t row, int lane) {
        const T* from = a.total + row * a.ldt;
        const int shift = shift_of(from);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift, end = row < a.rows ? a.cols - c : 0;
            load_part(t[k], from + c, end);
            load_part(dy[k], a.dy + row * a.lddy + c, end);
            if (MORE) load_part(more[k], a.dtotal + row * a.lddt + c, a.dtotal ? end : 0);
        }
        rstd = row < a.rows ? a.rstd[row] : 0.f;
    }
};

// As rms_backward_kernel, with rows off the boundaries (see rms_forward_shifted_kernel): a column's sum
// has its place in shared memory, where one lane or its neighbour adds to it.
template <typename T, typename W, int BLOCK>
__global__ void __launch_bounds__(BLOCK, backward_blocks_an_sm(BLOCK)) rms_backward_shifted_kernel(const RmsBackwardArgs<T, W> a) {
    constexpr bool kAhead = kBackwardAhead<BLOCK, T>, kMore = kBackwardMore<BLOCK>;
    extern __shared__ float room[];              // the weights; their gradients, of each group
    __shared__ float part[2][BLOCK / 32];
    const Columns places(a.lanes);
    const RowPlace<BLOCK> at(a.lanes);
    const int lane = at.lane, group = at.group, groups = at.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    float* const dgamma = room + places.size();
    for (int i = static_cast<int>(threadIdx.x); i < groups * places.size(); i += at.threads) dgamma[i] = 0.f;
    wait_for_previous_kernel();
    let_next_kernel_start();
    ShiftedRow<T, kMore> next;
    if (kAhead) next.load(a, static_cast<int64_t>(blockIdx.x) * groups + group, lane);
    place_weights(room, places, a.gamma, a.cols, a.lanes, at.threads);
    __syncthreads();
    const float* const weights = room + lane;
    float* const sums = dgamma + group * places.size() + lane;
    int turn = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        ShiftedRow<T, kMore> now;
        if constexpr (kAhead) {
            now = next;
            next.load(a, row + step, lane);
        } else {
            now.load(a, row, lane);
        }
        const int shift = shift_of(a.total + row * a.ldt);
        const auto hat_and_g = [&](int k, Pair (&hat)[4], Pair (&d)[4], Pair (&g)[4]) {
            now.t[k].get(hat);
            now.dy[k].get(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hat[i] = mul2(hat[i], Pair(now.rstd, now.rstd));
                g[i] = mul2(d[i], Pair(weights[places.at(2 * i - shift) + k * a.lanes], weights[places.at(2 * i + 1 - shift) + k * a.lanes]));
            }
        };
        Pair products(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift, end = row < a.rows ? a.cols - c : 0;
            keep_part(now.t[k], -c, end);
            keep_part(now.dy[k], -c, end);
            Pair hat[4], d[4], g[4];
            hat_and_g(k, hat, d, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                products = fma2(g[i], hat[i], products);
                float& lo = sums[places.at(2 * i - shift) + k * a.lanes];
                float& hi = sums[places.at(2 * i + 1 - shift) + k * a.lanes];
                fma2(d[i], hat[i], Pair(lo, hi)).get(lo, hi);
            }
        }
        // (all meet here: the next row's lanes add where this one's neighbours did)
        if (a.lanes <= 32) {
            __syncwarp();
        } else if (!a.dx) {
            __syncthreads();
        }
        if (!a.dx) continue;
        const float mean = row_sum<BLOCK>(both(products), a.lanes, part[turn]) / static_cast<float>(a.cols);
        turn ^= 1;
#pragma unroll
        for (int k = 0; k < kRowPacks; ++k) {
            const int c = 8 * (k * a.lanes + lane) - shift, end = row < a.rows ? a.cols - c : 0;
            Pair hat[4], d[4], g[4];
            hat_and_g(k, hat, d, g);
            if constexpr (!kMore) load_part(now.more[k], a.dtotal + row * a.lddt + c, a.dtotal ? end : 0);
            now.more[k].get(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = along_total(fma2(hat[i], Pair(-mean, -mean), g[i]), now.rstd, d[i], a.dtotal);
            }
            Eight<T> out;
            out.set(g);
            store_part(out, a.dx + row * a.lddx + c, -c, end, a.dx_along);
        }
    }
    if (!a.partial) return;
    __syncthreads();
    float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.cols;
    for (int c = static_cast<int>(threadIdx.x); c < a.cols; c += at.threads) {
        float sum = 0.f;
        for (int g = 0; g < groups; ++g) sum += dgamma[g * places.size() + places.at(c)];
        to[c] = sum;
    }
}

// Longer rows: dx, a row a block, twice over it.
template <typename T, typename W, bool WHOLE, bool OFF>
__global__ void __launch_bounds__(kMostRowLanes) rms_dx_wide_kernel(const RmsBackwardArgs<T, W> a) {
    __shared__ float part[kMostRowLanes / 32];
    const int64_t row = blockIdx.x;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const T* total = a.total + row * a.ldt;
    const T* dy = a.dy + row * a.lddy;
    const float rstd = a.rstd[row];
    float sum = 0.f;
    for (int c = first_column<WHOLE>(static_cast<int>(threadIdx.x)); c < a.cols; c += kMostRowLanes * 8) {
        Eight<T> t, g;
        Eight<W> w;
        t.template load<WHOLE>(total + c, a.cols - c);
        g.template load<WHOLE>(dy + c, a.cols - c);
        w.template load<WHOLE>(a.gamma + c, a.gamma ? a.cols - c : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(a.gamma ? g.get(i) * w.get(i) : g.get(i), t.get(i) * rstd, sum);
    }
    const float mean = row_sum<kMostRowLanes>(sum, kMostRowLanes, part) / static_cast<float>(a.cols);
    for (int c0 = 0; c0 < a.cols; c0 += kMostRowLanes * 8) {
        const int c = c0 + first_column<WHOLE>(static_cast<int>(threadIdx.x)), n = a.cols - c;
        if (!OFF && n <= 0) break;
        Eight<T> t, g, more;
        Eight<W> w;
        t.template load<WHOLE>(total + c, n);
        g.template load<WHOLE>(dy + c, n);
        w.template load<WHOLE>(a.gamma + c, a.gamma ? n : 0);
        more.template load<WHOLE>(a.dtotal + row * a.lddt + c, a.dtotal ? n : 0);
        Pair hat[4], v[4], by[4], d[4];
        t.get(hat);
        g.get(v);
        w.get(by);
        more.get(d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hat[i] = mul2(hat[i], Pair(rstd, rstd));
            if (a.gamma) v[i] = mul2(v[i], by[i]);
            v[i] = mul2(fma2(hat[i], Pair(-mean, -mean), v[i]), Pair(rstd, rstd));
            if (a.dtotal) v[i] = add2(v[i], d[i]);
        }
        g.set(v);
        store_result<WHOLE, OFF>(g, a.dx + row * a.lddx + c, n, kMostRowLanes);
    }
}

constexpr int kJoinThreads = 256;

// ... and gamma's gradient, 32 columns a block, its eight warps over the rows.
template <typename T, typename W>
__global__ void __launch_bounds__(kJoinThreads) rms_dgamma_wide_kernel(const RmsBackwardArgs<T, W> a, W* dgamma) {
    __shared__ float part[kJoinThreads / 32][32];
    const int lane = static_cast<int>(threadIdx.x) % 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    wait_for_previous_kernel();
    let_next_kernel_start();
    float sum = 0.f;
    if (c < a.cols) {
#pragma unroll 8
        for (int64_t row = warp; row < a.rows; row += kJoinThreads / 32)
            sum = fmaf(to_f32(a.dy[row * a.lddy + c]), to_f32(a.total[row * a.ldt + c]) * a.rstd[row], sum);
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= a.cols) return;
#pragma unroll
    for (int w = 1; w < kJoinThreads / 32; ++w) sum += part[w][lane];
    dgamma[c] = from_f32<W>(sum);
}

// The blocks' sums of a column, in their order.
template <typename W>
__global__ void __launch_bounds__(kJoinThreads) rms_dgamma_join_kernel(const float* partial, int blocks, int cols, W* dgamma) {
    __shared__ float part[kJoinThreads / 32][32];
    const int lane = static_cast<int>(threadIdx.x) % 32, warp = static_cast<int>(threadIdx.x) / 32;
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    wait_for_previous_kernel();
    let_next_kernel_start();
    float sum = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kJoinThreads / 32) sum += partial[static_cast<int64_t>(b) * cols + c];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
#pragma unroll
    for (int w = 1; w < kJoinThreads / 32; ++w) sum += part[w][lane];
    dgamma[c] = from_f32<W>(sum);
}

// ---------------------------------------------------------------- launches

// Whether rows of q lie as far from the 16-byte boundaries as p's (NULL: none there).
bool along(const void* p, int64_t ldp, const void* q, int64_t ldq, int bytes) {
    return !q || (((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) & 15u) == 0 && (ldp - ldq) * bytes % 16 == 0);
}
// Whether a row of few more lanes (a quarter at most) holds it wherever in an Eight it starts.
bool shiftable(int64_t cols) { return cols + 7 <= kRowColumns && row_lanes(cols + 7) * 4 <= row_lanes(cols) * 5; }

// Blocks of a forward launch: enough for every row, at most what the SMs hold at once.  Blocks of whole warps
// below their kernel's size find more room (896 threads of 72 registers), unless that puts more than 50 KB of
// rows with residuals on their way: 8192 x 5120 has 41 KB an SM, 16384 x 4096 with 48 KB takes 86 us and with
// 64 KB 91, 16384 x 2560 with 40 KB 53 and with 50 KB 58, rows of 4099 with 32 KB 117 and with 48 KB 85.
template <typename T, typename W>
int64_t forward_grid(const RmsForwardArgs<T, W>& a, bool quick, bool few, bool alone, int sms) {
    const int block = row_block(a.lanes), groups = block / a.lanes;
    int64_t most = forward_blocks_an_sm(block, sizeof(T), alone);
    if (sizeof(T) == 2 && quick && !alone && block > kSharedBlock) {
        most = std::max(896 / block, 1);
        if (few && a.residual) most = std::min<int64_t>(most, std::max(50000 / (4 * a.cols), 1));
    }
    return std::min((a.rows + groups - 1) / groups, sms * most);
}

template <typename T, typename W>
gemm_status_t forward_shifted(const RmsForwardArgs<T, W>& a, int sms, Queue queue) {
    return with_block(a.lanes, [&](auto block) {
        return launch<rms_forward_shifted_kernel<T, W, decltype(block)::value>>(forward_grid(a, true, true, false, sms), row_block(a.lanes),
                                                                                columns_bytes(a.lanes), queue, 1, a);
    });
}

// Shared memory of a gradient's shifted kernel.
constexpr size_t backward_room(int lanes) { return columns_bytes(lanes) * (1 + row_block(lanes) / lanes); }

template <typename T, typename W, bool Q8, bool WHOLE, bool OFF>
gemm_status_t forward(const RmsForwardArgs<T, W>& a, int sms, Queue queue) {
    if (a.cols > kRowColumns)
        return launch<rms_forward_wide_kernel<T, W, Q8, WHOLE, OFF>>(a.rows, kMostRowLanes, 0, queue, 1, a);
    const auto go = [&](auto block) {
        constexpr int kBlock = decltype(block)::value;
        // (without a residual there is not enough on its way: 8192 x 8192 bf16 55 us with 768 threads an SM, 45
        // with 1024; blocks of 257 to 384 threads fit twice either way)
        if constexpr (sizeof(T) == 2 && WHOLE && !Q8 && !OFF && kBlock != 384) {
            if (!a.residual)
                return launch<rms_forward_kernel<T, W, kBlock, Q8, WHOLE, true, OFF>>(forward_grid(a, WHOLE, !Q8, true, sms),
                                                                                      row_block(a.lanes), 0, queue, 1, a);
        }
        return launch<rms_forward_kernel<T, W, kBlock, Q8, WHOLE, false, OFF>>(forward_grid(a, WHOLE, !Q8, false, sms),
                                                                               row_block(a.lanes), 0, queue, 1, a);
    };
    if constexpr (OFF) return with_block_off(a.lanes, go);
    return with_block(a.lanes, go);
}
// whole: the inputs' rows (all on the boundaries, whole packs), off: a result's are not.
template <typename T, typename W, bool Q8>
gemm_status_t forward(const RmsForwardArgs<T, W>& a, bool whole, bool off, int sms, Queue queue) {
    if (!whole) return forward<T, W, Q8, false, false>(a, sms, queue);
    return off ? forward<T, W, Q8, true, true>(a, sms, queue) : forward<T, W, Q8, true, false>(a, sms, queue);
}

// Shared memory of the weight's gradient of a block's threads.
constexpr size_t sums_bytes(int block) { return static_cast<size_t>(block) * kLaneColumns * sizeof(float); }

// Blocks of a backward launch: enough for every row, at most what the SMs hold at once.
int64_t backward_grid(int64_t rows, int lanes, int sms) {
    const int block = row_block(lanes), groups = block / lanes;
    const int64_t blocks = (rows + groups - 1) / groups, most = static_cast<int64_t>(sms) * backward_blocks_an_sm(block);
    return blocks < most ? blocks : most;
}

template <typename T, typename W, bool WHOLE, bool OFF>
gemm_status_t backward(const RmsBackwardArgs<T, W>& a, int64_t grid, Queue queue) {
    const auto go = [&](auto block) {
        constexpr int kBlock = decltype(block)::value;
        const bool shared = kSharedBlock > a.lanes || !kBackwardRoom<kBlock, T>;
        return launch<rms_backward_kernel<T, W, kBlock, WHOLE, OFF>>(grid, row_block(a.lanes), shared ? sums_bytes(kBlock) : 0, queue, 1, a);
    };
    if constexpr (OFF) return with_block_off(a.lanes, go);
    return with_block(a.lanes, go);
}

template <typename T, typename W>
gemm_status_t backward_shifted(const RmsBackwardArgs<T, W>& a, int64_t grid, Queue queue) {
    return with_block(a.lanes, [&](auto block) {
        return launch<rms_backward_shifted_kernel<T, W, decltype(block)::value>>(grid, row_block(a.lanes), backward_room(a.lanes),
                                                                                 queue, 1, a);
    });
}

template <typename F>
gemm_status_t with_types(const gemm_rms_plan* p, F f) {
    return with_elem(p->elem, [&](auto t) {
        if (p->weight_elem == GEMM_ELEM_F32) return f(t, float());
        return f(t, t);
    });
}

// Lets the kernels of long rows have the shared memory that they ask for.
template <auto KERNEL>
bool allow(size_t bytes) {
    return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) == cudaSuccess;
}
template <typename T, typename W>
gemm_status_t prepare() {
    const auto wide = [](auto block) {
        constexpr int kBlock = decltype(block)::value;
        return allow<rms_backward_kernel<T, W, kBlock, true, false>>(sums_bytes(kBlock)) &&
               allow<rms_backward_kernel<T, W, kBlock, false, false>>(sums_bytes(kBlock)) &&
               allow<rms_backward_shifted_kernel<T, W, kBlock>>(backward_room(kBlock));
    };
    bool ok = wide(std::integral_constant<int, 768>()) && wide(std::integral_constant<int, kMostRowLanes>()) &&
              allow<rms_backward_kernel<T, W, kMostRowLanes, true, true>>(sums_bytes(kMostRowLanes)) &&
              allow<rms_backward_shifted_kernel<T, W, 384>>(backward_room(384)) &&
              allow<rms_backward_shifted_kernel<T, W, 512>>(backward_room(512));
    if constexpr (sizeof(T) == 2)
        ok = ok && allow<rms_forward_shifted_kernel<T, W, 768>>(columns_bytes(768)) &&
             allow<rms_forward_shifted_kernel<T, W, kMostRowLanes>>(columns_bytes(kMostRowLanes));
    if (ok) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

gemm_status_t check_forward(const gemm_rms_plan* p, int64_t rows, const void* x, int64_t ldx, const void* residual,
                            int64_t ldr, const void* gamma, float eps, const void* total, int64_t ldt, const void* out,
                            int64_t ldo, const float* rstd) {
    if (!p || rows < 0 || rows > p->max_rows || !(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !out || ldx < p->cols || ldo < p->cols || (residual && ldr < p->cols) ||
                     (total && (ldt < p->cols || total == out))))
        return GEMM_ERR_INVALID_ARG;
    const int e = elem_bytes(p->elem);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(total, e) || !aligned(gamma, elem_bytes(p->weight_elem)) ||
        !aligned(rstd, 4))
        return GEMM_ERR_ALIGNMENT;
    return check_device(p->device);
}

}  // namespace
}  // namespace gbt

extern "C" {

gemm_status_t gemm_rms_plan_create(int64_t max_rows, int64_t cols, gemm_elem_t elem, gemm_elem_t weight_elem,
                                   gemm_rms_plan_t* plan) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!gbt::valid_elem(elem) || (weight_elem != elem && weight_elem != GEMM_ELEM_F32)) return GEMM_ERR_UNSUPPORTED;
    if (max_rows < 0 || max_rows > INT32_MAX || cols < 1 || cols > gbt::kMostColumns) return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    const gemm_status_t st = gbt::begin_plan(&device, &sms);
    if (st != GEMM_OK) return st;
    size_t sums = 0;
    if (cols <= gbt::kRowColumns)
        sums = static_cast<size_t>(gbt::backward_grid(max_rows, gbt::row_lanes(cols), sms) * cols) * sizeof(float);
    void* memory = nullptr;
    const gemm_status_t room = sums > 0 ? gbt::allocate(&memory, sums) : GEMM_OK;
    if (room != GEMM_OK) return room;
    gemm_rms_plan* p = new (std::nothrow) gemm_rms_plan();
    if (!p) {
        cudaFree(memory);
        return GEMM_ERR_OOM;
    }
    p->max_rows = max_rows;
    p->cols = cols;
    p->elem = elem;
    p->weight_elem = weight_elem;
    p->device = device;
    p->num_sms = sms;
    p->partial = static_cast<float*>(memory);
    const gemm_status_t ready = gbt::with_types(p, [](auto t, auto v) { return gbt::prepare<decltype(t), decltype(v)>(); });
    if (ready != GEMM_OK) {
        gemm_rms_plan_destroy(p);
        return ready;
    }
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_rms_forward(gemm_rms_plan_t p, int64_t rows, const void* x, int64_t ldx, const void* residual,
                               int64_t ldr, const void* gamma, float eps, void* total, int64_t ldt, void* y,
                               int64_t ldy, float* rstd, void* stream) {
    const gemm_status_t st = gbt::check_forward(p, rows, x, ldx, residual, ldr, gamma, eps, total, ldt, y, ldy, rstd);
    if (st != GEMM_OK) return st;
    const int e = gbt::elem_bytes(p->elem);
    if (!gbt::aligned(y, e)) return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    // (the inputs alone decide which kernel sums their rows, and in which order: the same numbers wherever results go)
    const bool whole = p->cols % 8 == 0 && gbt::rows_aligned(x, ldx, e) && gbt::packs_aligned(residual, ldr, e) &&
                       gbt::aligned(gamma, 16);
    const bool shifted = !whole && gbt::shiftable(p->cols) && gbt::along(x, ldx, residual, ldr, e);
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        const gbt::RmsForwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const T*>(residual),
                                          static_cast<const W*>(gamma), static_cast<T*>(total), static_cast<T*>(y), nullptr,
                                          nullptr, rstd, ldx, ldr, ldt, ldy, 0, 0, rows, eps, static_cast<int>(p->cols),
                                          gbt::row_lanes(p->cols + (shifted && sizeof(T) == 2 ? 7 : 0)), gbt::along(x, ldx, total, ldt, e),
                                          gbt::along(x, ldx, y, ldy, e)};
        const gbt::Queue queue{stream, p->device};
        if constexpr (sizeof(T) == 2) {
            if (shifted) return gbt::forward_shifted<T, W>(a, p->num_sms, queue);
        }
        return gbt::forward<T, W, false>(a, whole, !a.total_along || !a.y_along, p->num_sms, queue);
    });
}

gemm_status_t gemm_rms_forward_fp8(gemm_rms_plan_t p, int64_t rows, const void* x, int64_t ldx, const void* residual,
                                   int64_t ldr, const void* gamma, float eps, void* total, int64_t ldt, void* q,
                                   int64_t ldq, float* scales, int64_t lds, float* rstd, void* stream) {
    const gemm_status_t st = gbt::check_forward(p, rows, x, ldx, residual, ldr, gamma, eps, total, ldt, q, ldq, rstd);
    if (st != GEMM_OK) return st;
    if (rows > 0 && (!scales || lds < gbt::groups_of(p->cols))) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(scales, 4)) return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    const int e = gbt::elem_bytes(p->elem);
    const bool whole = p->cols % 8 == 0 && gbt::rows_aligned(x, ldx, e) && gbt::packs_aligned(residual, ldr, e) &&
                       gbt::aligned(gamma, 16);
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        const gbt::RmsForwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const T*>(residual),
                                          static_cast<const W*>(gamma), static_cast<T*>(total), nullptr,
                                          static_cast<uint8_t*>(q), scales, rstd, ldx, ldr, ldt, 0, ldq, lds, rows, eps,
                                          static_cast<int>(p->cols), gbt::row_lanes(p->cols), gbt::along(x, ldx, total, ldt, e), false};
        const gbt::Queue queue{stream, p->device};
        return gbt::forward<T, W, true>(a, whole, !a.total_along || !gbt::bytes_aligned(q, ldq), p->num_sms, queue);
    });
}

gemm_status_t gemm_rms_backward(gemm_rms_plan_t p, int64_t rows, const void* total, int64_t ldt, const void* gamma,
                                const float* rstd, const void* dy, int64_t lddy, const void* dtotal, int64_t lddt,
                                void* dx, int64_t lddx, void* dgamma, void* stream) {
    if (!p || rows < 0 || rows > p->max_rows) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!total || !rstd || !dy || ldt < p->cols || lddy < p->cols || (dtotal && lddt < p->cols) ||
                     (dx && lddx < p->cols)))
        return GEMM_ERR_INVALID_ARG;
    const int e = gbt::elem_bytes(p->elem), w = gbt::elem_bytes(p->weight_elem);
    if (!gbt::aligned(total, e) || !gbt::aligned(dy, e) || !gbt::aligned(dtotal, e) || !gbt::aligned(dx, e) ||
        !gbt::aligned(gamma, w) || !gbt::aligned(dgamma, w) || !gbt::aligned(rstd, 4))
        return GEMM_ERR_ALIGNMENT;
    const gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK || (!dx && !dgamma)) return st;
    const bool whole = p->cols % 8 == 0 && gbt::rows_aligned(total, ldt, e) && gbt::rows_aligned(dy, lddy, e) &&
                       gbt::packs_aligned(dtotal, lddt, e) && gbt::aligned(gamma, 16);
    // (a result's place decides nothing but its stores: the same numbers wherever it goes)
    const bool shifted = !whole && gbt::shiftable(p->cols) && gbt::along(total, ldt, dy, lddy, e) &&
                         gbt::along(total, ldt, dtotal, lddt, e);
    const gbt::Queue queue{stream, p->device};
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        const int cols = static_cast<int>(p->cols), lanes = gbt::row_lanes(cols + (shifted ? 7 : 0));
        const unsigned tiles = static_cast<unsigned>((p->cols + 31) / 32);
        const gbt::RmsBackwardArgs<T, W> a{static_cast<const T*>(total), static_cast<const W*>(gamma), rstd,
                                           static_cast<const T*>(dy), static_cast<const T*>(dtotal), static_cast<T*>(dx),
                                           dgamma ? p->partial : nullptr, ldt, lddy, lddt, lddx, rows, cols, lanes,
                                           gbt::along(total, ldt, dx, lddx, e)};
        gemm_status_t s = GEMM_OK;
        if (cols > gbt::kRowColumns) {
            // (the weight's gradient first: dx may overwrite dy or total)
            if (dgamma)
                s = gbt::launch<gbt::rms_dgamma_wide_kernel<T, W>>(tiles, gbt::kJoinThreads, 0, queue, 1, a,
                                                                    static_cast<W*>(dgamma));
            if (s == GEMM_OK && dx && rows > 0)
                s = !whole         ? gbt::launch<gbt::rms_dx_wide_kernel<T, W, false, false>>(rows, gbt::kMostRowLanes, 0, queue, 1, a)
                    : a.dx_along ? gbt::launch<gbt::rms_dx_wide_kernel<T, W, true, false>>(rows, gbt::kMostRowLanes, 0, queue, 1, a)
                                 : gbt::launch<gbt::rms_dx_wide_kernel<T, W, true, true>>(rows, gbt::kMostRowLanes, 0, queue, 1, a);
            return s;
        }
        const int64_t grid = gbt::backward_grid(rows, lanes, p->num_sms);
        if (grid > 0)
            s = shifted ? gbt::backward_shifted<T, W>(a, grid, queue)
                : !whole     ? gbt::backward<T, W, false, false>(a, grid, queue)
                : a.dx_along ? gbt::backward<T, W, true, false>(a, grid, queue)
                             : gbt::backward<T, W, true, true>(a, grid, queue);
        if (s == GEMM_OK && dgamma)
            s = gbt::launch<gbt::rms_dgamma_join_kernel<W>>(tiles, gbt::kJoinThreads, 0, queue, 1, p->partial,
                                                            static_cast<int>(grid), cols, static_cast<W*>(dgamma));
        return s;
    });
}

gemm_status_t gemm_rms_plan_destroy(gemm_rms_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->partial) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
