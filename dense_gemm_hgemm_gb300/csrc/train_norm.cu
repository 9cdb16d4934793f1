// train_norm.cu -- layer norm of gemm_train.h, forward and backward.
#include <new>

#include "train_common.cuh"

struct gemm_norm_plan {
    int64_t max_rows, cols;
    gemm_elem_t elem, weight_elem;
    int device, num_sms;
    void* memory;        // one allocation: the error word and `partial`
    int32_t* error_word;
    float* partial;      // [2][blocks][cols] sums of the weight gradients
    gbt::Waits waits;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;      // of the kernels that loop over a row or a column
constexpr int kMaxLanes = 1024;
constexpr int kLaneCols = 16;      // columns a lane keeps in registers
constexpr int kPairs = kLaneCols / 2;

// ---- rows in registers ----------------------------------------------------------
//
// `lanes` threads (4 to 1024, a power of two) keep one row, kLaneCols columns each:
// PACKS packs of VEC elements, pack k of lane l at column (k * lanes + l) * VEC.  A
// block has BLOCK / lanes such groups, each with its own rows, and asks for its next
// row before it works on the present one.  So a row is read once, and its statistics
// are exact two-pass ones at no further traffic.  These kernels serve few rows (1 x 4096:
// 2.8 us, the latency of a launch, a load and two sums) and rows too short for a copy each
// (65536 x 64 bf16: forward 9.3 us, backward 12.5).

// WHOLE: the row's length is a multiple of VEC, so a pack is in it or not.
template <typename T, int VEC, int COLS, bool WHOLE>
struct RowPacks {
    static constexpr int PACKS = COLS / VEC;
    Pack<T, VEC> p[PACKS];
    __device__ __forceinline__ void load(const T* row, int lane, int lanes, int cols) {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (WHOLE && c >= cols) {
                p[k].clear();
            } else {
                p[k] = load_pack<T, VEC>(row + c, WHOLE ? VEC : cols - c);
            }
        }
    }
    __device__ __forceinline__ void store(T* row, int lane, int lanes, int cols) const {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (!WHOLE || c < cols) store_pack<T, VEC>(row + c, WHOLE ? VEC : cols - c, p[k]);
        }
    }
};

// A lane's columns of a weight vector (`other` without one, and past the row's end).
template <typename W, int VEC, int COLS>
__device__ __forceinline__ void load_weights(const W* w, float other, int lane, int lanes, int cols, Pair (&v)[COLS / 2]) {
    float f[COLS];
#pragma unroll
    for (int k = 0; k < COLS / VEC; ++k) {
        const int c = (k * lanes + lane) * VEC;
        float part[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) part[i] = other;
        if (w) load_values<W, VEC>(w + c, cols - c, part);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[k * VEC + i] = part[i];
    }
#pragma unroll
    for (int j = 0; j < COLS / 2; ++j) v[j] = Pair(f[2 * j], f[2 * j + 1]);
}

template <int N>
__device__ __forceinline__ float sum_of(const Pair (&v)[N]) {
    Pair s = add2(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < N; ++j) s = add2(s, v[j]);
    float lo, hi;
    s.get(lo, hi);
    return lo + hi;
}

__device__ __forceinline__ float half_sum(float v) {     // over 16 lanes
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums over a group, in every lane: shuffles in the warp, then one exchange in shared
// memory behind the group's own barrier.  Two exchange buffers in turn: a warp that is
// a sum ahead has passed the barrier that the others reach only after their reads.
template <int N>
struct GroupSum {
    float (*part)[N][32];    // [2][N][32] of the group (where it is more than a warp)
    int lanes, barrier, turn;
    // the lanes of a group within a warp, which other groups share
    __device__ __forceinline__ float few(float v) const {
        const unsigned mask = ((1u << lanes) - 1u) << (threadIdx.x % 32 / lanes * lanes);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            if (o < lanes) v += __shfl_xor_sync(mask, v, o);
        return v;
    }
    __device__ __forceinline__ void meet() {
        asm volatile("bar.sync %0, %1;" :: "r"(barrier), "r"(lanes) : "memory");
    }
    __device__ __forceinline__ void operator()(float (&v)[N], int lane) {
        const int warps = lanes / 32, l = lane % 32;
        if (lanes <= 32) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = lanes == 32 ? warp_sum(v[i]) : few(v[i]);
            return;
        }
        if constexpr (N == 1) {
            v[0] = warp_sum(v[0]);
            if (l == 0) part[turn][0][lane / 32] = v[0];
            meet();
            v[0] = l < warps ? part[turn][0][l] : 0.f;
            if (warps > 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
            if (warps > 8) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
            if (warps > 4) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
            if (warps <= 16) v[0] = __shfl_sync(0xffffffffu, v[0], 0);
        } else {
            // two values share the steps: half the lanes go on with one, half with the other
            const bool upper = l >= 16;
            float mine = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
            mine = half_sum(mine);
            if ((l & 15) == 0) part[turn][upper][lane / 32] = mine;
            meet();
            const int w = l & 15;
            mine = w < warps ? part[turn][upper][w] : 0.f;
            if (warps > 16) mine += w + 16 < warps ? part[turn][upper][w + 16] : 0.f;
            mine = half_sum(mine);
            v[0] = __shfl_sync(0xffffffffu, mine, 0);
            v[1] = __shfl_sync(0xffffffffu, mine, 16);
        }
        turn ^= 1;
    }
};

// Forward, once a row is in the lanes' pairs: subtracts its mean (columns past the row's
// end stay zero) and returns it;
template <int VEC, int N>
__device__ __forceinline__ float centre(Pair (&v)[N], GroupSum<1>& sum, float inverse_n, bool full, int lane, int lanes,
                                        int cols) {
    float s[1] = {sum_of(v)};
    sum(s, lane);
    const float mu = s[0] * inverse_n;
    const Pair minus(-mu, -mu);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = add2(v[j], minus);
    if (!full) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (2 * j / VEC * lanes + lane) * VEC + 2 * j % VEC;
            const int c1 = VEC == 1 ? c + lanes : c + 1;
            float lo, hi;
            v[j].get(lo, hi);
            v[j] = Pair(c < cols ? lo : 0.f, c1 < cols ? hi : 0.f);
        }
    }
    return mu;
}

// then 1 / sqrt(variance + eps);
template <int N>
__device__ __forceinline__ float rstd_of(const Pair (&v)[N], GroupSum<1>& sum, float inverse_n, float eps, int lane) {
    Pair square = mul2(v[0], v[0]);
#pragma unroll
    for (int j = 1; j < N; ++j) square = fma2(v[j], v[j], square);
    float lo, hi, s[1];
    square.get(lo, hi);
    s[0] = lo + hi;
    sum(s, lane);
    return rsqrtf(s[0] * inverse_n + eps);
}

// Weights in shared memory.  Packs of eight fp32 values are kept as two halves, each with
// the others' halves, so that neighbouring lanes' 16-byte reads are neighbours (side by side
// they would share banks: 61 us instead of 46 at 16384 x 4096 with fp32 weights).
template <typename W, int VEC>
struct Staged {
    static constexpr bool kHalves = VEC * sizeof(W) > 16;
    static constexpr int kPer = kHalves ? VEC / 2 : VEC;
    W* at;
    int half;                // elements of a half: those of the row's packs
    __device__ __forceinline__ void put(int c, W v) {
        at[kHalves ? (c % VEC / kPer) * half + c / VEC * kPer + c % kPer : c] = v;
    }
    __device__ __forceinline__ void get(int c, float (&v)[VEC]) const {      // the pack at column c
#pragma unroll
        for (int h = 0; h < VEC / kPer; ++h) {
            const Pack<W, kPer> q = load_pack<W, kPer>(at + (kHalves ? h * half + c / VEC * kPer : c), kPer);
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[h * kPer + i] = q.get(i);
        }
    }
};

// and the result, with the weights read on the way, a pack at a time to store(column, pack)
// (single elements: to y).
template <typename T, typename W, int VEC, int N, typename F>
__device__ __forceinline__ void normalise(const Pair (&v)[N], float r, const Staged<W, VEC>& gamma,
                                          const Staged<W, VEC>& beta, T* y, int lane, int lanes, int cols, F store) {
    const Pair r2(r, r);
    if constexpr (VEC == 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = 2 * j * lanes + lane, c1 = c + lanes;
            float g0[1], g1[1], b0[1], b1[1], lo, hi;
            gamma.get(c, g0);                            // (there is room for all lanes' columns)
            gamma.get(c1, g1);
            beta.get(c, b0);
            beta.get(c1, b1);
            fma2(mul2(v[j], r2), Pair(g0[0], g1[0]), Pair(b0[0], b1[0])).get(lo, hi);
            if (c < cols) y[c] = from_f32<T>(lo);
            if (c1 < cols) y[c1] = from_f32<T>(hi);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2 * N / VEC; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c >= cols) break;
            float g[VEC], b[VEC];
            gamma.get(c, g);
            beta.get(c, b);
            Pack<T, VEC> out;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
                set_pair(out, i,
                         fma2(mul2(v[k * (VEC / 2) + i], r2), Pair(g[2 * i], g[2 * i + 1]), Pair(b[2 * i], b[2 * i + 1])));
            store(c, out);
        }
    }
}

template <typename T, typename W>
struct ForwardArgs {
    const T* x;
    const W* gamma;
    const W* beta;
    T* y;
    float* mean;
    float* rstd;
    int32_t* error;
    int64_t ldx, ldy, rows;
    float eps;
    int cols, lanes;
    Waits waits;
};

// KEEP: gamma and beta stay in registers over the rows (else they are read for each
// row, where the block's registers would not suffice).
template <typename T, typename W, int VEC, int BLOCK, bool KEEP>
__global__ void __launch_bounds__(BLOCK) norm_forward_kernel(const ForwardArgs<T, W> a) {
    __shared__ float part[BLOCK / 32][2][1][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lanes = a.lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (BLOCK / lanes);
    int64_t row = static_cast<int64_t>(blockIdx.x) * (BLOCK / lanes) + group;
    if (row >= a.rows) return;
    const bool full = a.cols == lanes * kLaneCols;
    GroupSum<1> sum{part[group % (BLOCK / 32)], lanes, 1 + group, 0};
    RowPacks<T, VEC, kLaneCols, false> next;
    next.load(a.x + row * a.ldx, lane, lanes, a.cols);
    Pair gamma[kPairs], beta[kPairs];
    if (KEEP) {
        load_weights<W, VEC, kLaneCols>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
        load_weights<W, VEC, kLaneCols>(a.beta, 0.f, lane, lanes, a.cols, beta);
    }
    const float inverse_n = 1.f / static_cast<float>(a.cols);
    for (; row < a.rows; row += step) {
        Pair v[kPairs];
        to_pairs(next.p, v);                     // (columns past the row's end are zeros)
        if (row + step < a.rows) next.load(a.x + (row + step) * a.ldx, lane, lanes, a.cols);
        const float mu = centre<VEC>(v, sum, inverse_n, full, lane, lanes, a.cols);
        const float r = rstd_of(v, sum, inverse_n, a.eps, lane);
        if (!KEEP) {
            load_weights<W, VEC, kLaneCols>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
            load_weights<W, VEC, kLaneCols>(a.beta, 0.f, lane, lanes, a.cols, beta);
        }
        const Pair r2(r, r);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = fma2(mul2(v[j], r2), gamma[j], beta[j]);
        RowPacks<T, VEC, kLaneCols, false> out;
        from_pairs(v, out.p);
        out.store(a.y + row * a.ldy, lane, lanes, a.cols);
        if (lane == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
}

// ---- rows through rings ------------------------------------------------------------
//
// Many rows: one block an SM, in which each group has a ring of stages in shared memory
// and brings its next rows there by bulk copies.  The barrier of the group's first sum
// tells that all lanes have read a stage, so its first lane asks for the next row right
// behind it; there is no copying warp and no second barrier.  The bytes in flight do not
// depend on how many registers are left for loads: the register kernels keep 24 KB an SM
// in flight at 16384 x 4096, the rings over 100 KB.  Forward is bound by bytes: 16384 x 4096
// bf16 44.5 us, 0.90 of the copy bandwidth (in registers 64), fp32 87 us, 0.92; 65536 x 1000
// 44 us, 0.89; 4096 x 16384 45 us, 0.88.  Backward does four sums' work an element (two of the row, two of
// the columns) with 512 threads of 125 registers, and is bound by issuing that and by the
// one barrier a row that nothing overlaps: 8192 x 8192 77 us, 0.78 (80 where each of the two
// sums took its own shuffles; 82 in registers); fp32 138 us, 0.87.

constexpr int kRingRows = 1 << 30;         // rows are counted in 32 bits there, some steps beyond the last
constexpr int kRingSlots = 64;             // stages of a block, at most
constexpr int kRingShared = 208 * 1024;    // its dynamic shared memory, at most
constexpr int kForwardRing = 1024;         // threads of the blocks
constexpr int kBackwardRing = 512;

// A block's waits: ns that one may last (0: one ran out, nothing waits long any more), and
// bytes that a stage waits for beyond its copies.
struct RingWaits {
    uint32_t patience, limit, extra;
};

// A group's ring; each stage holds a row from each of N sources.  Where rows do not begin or
// end at 16-byte boundaries (ANY), the whole 16-byte units around a row are copied; the first
// and the last row of the matrix, whose units may reach beyond it, are left to plain loads.
template <int N, bool ANY>
struct Ring {
    uint8_t* memory;
    uint64_t* full;
    RingWaits* waits;
    int32_t* error;
    const uint8_t* src[N];
    int64_t stride[N];                     // bytes
    int rows, step;                        // the matrix' rows; from one of the group's to its next
    int row_bytes, stage_bytes, stages;    // (stage_bytes: of one source)
    Turn turn;
    int asked;                             // rows asked for, by the lane that asks

    __device__ __forceinline__ bool direct(int row) const { return ANY && (row == 0 || row == rows - 1); }
    __device__ __forceinline__ void ask(int stage, int row) {
        if (is_dead(&waits->patience)) return;
        ++asked;
        if (direct(row)) {
            expect_bytes(&full[stage], waits->extra);
            return;
        }
        const uint8_t* from[N];
        uint32_t bytes[N], all = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            from[k] = src[k] + row * stride[k];
            bytes[k] = static_cast<uint32_t>(row_bytes);
            if (ANY) {
                const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from[k]) & 15u);
                from[k] -= off;
                bytes[k] = (off + bytes[k] + 15u) / 16u * 16u;
            }
            all += bytes[k];
        }
        expect_bytes(&full[stage], all + waits->extra);
#pragma unroll
        for (int k = 0; k < N; ++k) copy_bytes(memory + (stage * N + k) * stage_bytes, from[k], bytes[k], &full[stage]);
    }
    // (one lane)
    __device__ __forceinline__ void begin(int row) {
        for (int k = 0; k < stages && row < rows; ++k, row += step) ask(k, row);
    }
    __device__ __forceinline__ void wait() const { wait_or_die(&full[turn.at], turn.round & 1, &waits->patience, error); }
    // Source k's row, in the present stage (or in the matrix), once waited for.
    __device__ __forceinline__ const uint8_t* at(int k, int row) const {
        const uint8_t* from = src[k] + row * stride[k];
        if (direct(row)) return from;
        return memory + (turn.at * N + k) * stage_bytes + (ANY ? reinterpret_cast<uintptr_t>(from) & 15u : 0);
    }
    // All lanes have read that stage: the row, `stages` steps on from what it held.  (The warp
    // goes on together: without the __syncwarp its first lane took the rest of the row by
    // itself, twice the instructions.)
    __device__ __forceinline__ void refill(int lane, int stage, int row) {
        if (lane == 0 && row < rows) ask(stage, row);
        __syncwarp();
    }
    // After a wait that ran out (one lane): what was asked for may still come.
    __device__ __forceinline__ void end() const {
        if (!is_dead(&waits->patience)) return;
        const uint32_t began = timer_ns();
        for (int k = asked > stages ? asked - stages : 0; k < asked; ++k)
            wait_until(&full[k % stages], (k / stages) & 1, began, waits->limit);
    }
};

// Bytes of a row in a stage.
__host__ __device__ constexpr int ring_stage_bytes(int row_bytes, bool any) {
    return any ? (row_bytes + 15) / 16 * 16 + 16 : row_bytes;
}

struct RingBarriers {
    uint64_t full[kRingSlots];
    RingWaits waits;
};

// (one thread)
__device__ __forceinline__ void init_ring(RingBarriers& ring, int slots, const Waits& waits) {
    for (int k = 0; k < slots; ++k) init_barrier(&ring.full[k], 1);
    ring.waits = {waits.limit, waits.limit, waits.extra_bytes()};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Rows off the 16-byte boundaries, in packs all the same: a pack is a 16-byte unit of the
// memory, from the one that the row begins in, so the row's elements stand at the positions
// off .. end - 1 from there.  A block's rows are multiples of gridDim.x rows apart, which has to
// be a multiple of 16 bytes (152 rows are), so they share `off` and a lane keeps its columns; and
// what is read and what is written have the same `off` (else single elements move).  Warps
// with the row's ends take more steps for them.  10000 x 5003 bf16: forward 51 us, backward
// 110; with single elements 71 and 160; rows of 5008 take 40 and 75.
template <int VEC>
struct Span {
    int off, end;
    __device__ __forceinline__ bool holds(int p) const { return p >= off && p + VEC <= end; }     // a whole pack
    __device__ __forceinline__ bool has(int p) const { return p >= off && p < end; }
    // all packs of a warp's lanes
    __device__ __forceinline__ bool holds_all(int lane, int lanes, int packs) const {
        return __all_sync(0xffffffffu, lane * VEC >= off && ((packs - 1) * lanes + lane + 1) * VEC <= end);
    }
    // A row's packs; `unguarded`: the units around it may be read.
    template <typename T, int PACKS>
    __device__ __forceinline__ void load(Pack<T, VEC> (&q)[PACKS], const T* row, bool unguarded, int lane, int lanes) const {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int p = (k * lanes + lane) * VEC;
            if (p >= end) {
                q[k].clear();
            } else if (unguarded || holds(p)) {
                q[k] = load_pack<T, VEC>(row + (p - off), VEC);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[k].set_raw(i, has(p + i) ? row[p - off + i] : from_f32<T>(0.f));
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, int p, const Pack<T, VEC>& q) const {
        if (holds(p)) {
            store_pack<T, VEC>(row + (p - off), VEC, q);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (has(p + i)) row[p - off + i] = reinterpret_cast<const T*>(&q.raw)[i];
        }
    }
    // Zeros where the row has no elements.
    template <int N>
    __device__ __forceinline__ void clear(Pair (&v)[N], int lane, int lanes) const {
#pragma unroll
        for (int k = 0; k < 2 * N / VEC; ++k) {
            const int p = (k * lanes + lane) * VEC;
            if (holds(p)) continue;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                float lo, hi;
                v[k * (VEC / 2) + i].get(lo, hi);
                v[k * (VEC / 2) + i] = Pair(has(p + 2 * i) ? lo : 0.f, has(p + 2 * i + 1) ? hi : 0.f);
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ int off_of_row(const T* base, int64_t ld, int64_t row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(base + row * ld) & 15u) / sizeof(T));
}

// gamma and beta wait in shared memory behind the rings.  COLS columns a lane: with 32 a row
// takes half the warps of 16, and so half the work that does not depend on its length.
template <typename T, typename W, int VEC, int COLS, bool SHIFT>
__global__ void __launch_bounds__(kForwardRing, 1) norm_forward_ring_kernel(const ForwardArgs<T, W> a, int stages) {
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ RingBarriers barriers;
    __shared__ float part[kForwardRing / 32][2][1][32];
    const int lanes = a.lanes, groups = kForwardRing / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    constexpr bool kAny = VEC == 1 || SHIFT;
    const int row_bytes = a.cols * static_cast<int>(sizeof(T)), stage_bytes = ring_stage_bytes(row_bytes, kAny);
    Staged<W, VEC> gamma{reinterpret_cast<W*>(memory + groups * stages * stage_bytes), lanes * COLS / 2};
    Staged<W, VEC> beta{gamma.at + lanes * COLS, gamma.half};
    if (threadIdx.x == 0) init_ring(barriers, groups * stages, a.waits);
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    // (threads behind the last whole group have no rows)
    int row = group < groups ? static_cast<int>(blockIdx.x + group * gridDim.x) : static_cast<int>(a.rows);
    Ring<1, kAny> ring{memory + group * stages * stage_bytes,
                 barriers.full + group * stages,
                 &barriers.waits,
                 a.error,
                 {reinterpret_cast<const uint8_t*>(a.x)},
                 {a.ldx * static_cast<int64_t>(sizeof(T))},
                 static_cast<int>(a.rows),
                 static_cast<int>(groups * gridDim.x),
                 row_bytes,
                 stage_bytes,
                 stages,
                 {0, 0},
                 0};
    if (lane == 0 && group < groups) ring.begin(row);
    const int off = SHIFT ? off_of_row(a.x, a.ldx, blockIdx.x) : 0;
    for (int c = threadIdx.x; c < a.cols; c += kForwardRing) {
        gamma.put(c + off, a.gamma ? a.gamma[c] : from_f32<W>(1.f));
        beta.put(c + off, a.beta ? a.beta[c] : from_f32<W>(0.f));
    }
    __syncthreads();
    const Span<VEC> span{off, off + a.cols};
    const bool inner = SHIFT && span.holds_all(lane, lanes, COLS / VEC);
    const bool full = a.cols == lanes * COLS;
    const float inverse_n = 1.f / static_cast<float>(a.cols);
    GroupSum<1> sum{part[group], lanes, group, 0};       // (barrier 0 is free from here on)
    T* y = a.y + row * a.ldy;
    const int64_t y_step = ring.step * a.ldy;
    for (; row < ring.rows; row += ring.step, y += y_step, ring.turn.next(1, stages)) {
        Pair v[COLS / 2];
        {
            RowPacks<T, VEC, COLS, true> in;
            ring.wait();
            const T* from = reinterpret_cast<const T*>(ring.at(0, row));
            if constexpr (SHIFT) {
                if (inner) {
                    in.load(from - off, lane, lanes, span.end);
                } else {
                    span.load(in.p, from, !ring.direct(row), lane, lanes);
                }
                to_pairs(in.p, v);
                if (!inner) span.clear(v, lane, lanes);
            } else {
                in.load(from, lane, lanes, a.cols);
                to_pairs(in.p, v);
            }
        }
        const float mu = centre<VEC>(v, sum, inverse_n, SHIFT || full, lane, lanes, a.cols);
        if (SHIFT && !inner) span.clear(v, lane, lanes);
        ring.refill(lane, ring.turn.at, row + stages * ring.step);
        const float r = rstd_of(v, sum, inverse_n, a.eps, lane);
        normalise<T, W, VEC>(v, r, gamma, beta, y, lane, lanes, span.end, [&](int p, const Pack<T, VEC>& q) {
            if (!SHIFT || inner) {
                store_pack<T, VEC>(y + (p - off), VEC, q);
            } else {
                span.store(y, p, q);
            }
        });
        if (lane == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
    if (lane == 0 && group < groups) ring.end();
}

template <typename T, typename W>
struct BackwardArgs {
    const T* x;
    const W* gamma;
    const float* mean;
    const float* rstd;
    const T* dy;
    T* dx;
    float* partial;      // [2][gridDim.x][cols]
    int32_t* error;
    int64_t ldx, lddy, lddx, rows;
    int cols, lanes;
    bool weights;        // dgamma or dbeta is wanted
    Waits waits;
};

// Backward, once xh and g are in the lanes' pairs: the group's sums, then dx.
__device__ __forceinline__ void row_sums(Pair sum_g, Pair sum_gx, GroupSum<2>& sum, int lane, float (&s)[2]) {
    float lo, hi;
    sum_g.get(lo, hi);
    s[0] = lo + hi;
    sum_gx.get(lo, hi);
    s[1] = lo + hi;
    sum(s, lane);
}

__device__ __forceinline__ void dx_of(const Pair (&hat)[kPairs], Pair (&g)[kPairs], const float (&s)[2], float inverse_n,
                                      Pair r2) {
    const float mean_g = s[0] * inverse_n, mean_gx = s[1] * inverse_n;
    const Pair minus_g(-mean_g, -mean_g), minus_gx(-mean_gx, -mean_gx);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) g[j] = mul2(r2, fma2(hat[j], minus_gx, add2(g[j], minus_g)));
}

template <typename T, int VEC, bool WHOLE>
__device__ __forceinline__ void write_dx(const Pair (&hat)[kPairs], Pair (&g)[kPairs], const float (&s)[2], float inverse_n,
                                         Pair r2, T* dx, int lane, int lanes, int cols) {
    dx_of(hat, g, s, inverse_n, r2);
    RowPacks<T, VEC, kLaneCols, WHOLE> out;
    from_pairs(g, out.p);
    out.store(dx, lane, lanes, cols);
}

// Sums kept as [2][kLaneCols][lanes] in shared memory, to the block's rows of the partial
// sums, in the order of the columns.
template <int VEC, int THREADS>
__device__ __forceinline__ void copy_partial(int lanes, int cols, const float* join, float* partial) {
    for (int which = 0; which < 2; ++which) {
        float* out = partial + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * cols;
        for (int c = threadIdx.x; c < cols; c += THREADS) {
            const int pack = c / VEC;                    // column c is element c % VEC of this pack
            out[c] = join[(which * kLaneCols + pack / lanes * VEC + c % VEC) * lanes + pack % lanes];
        }
    }
}

// The sums of a block's groups, joined in the order of the groups through shared memory
// (`join`: [groups][2][lanes * kLaneCols], group g's column c at c + off_of(g)), to its rows of
// the partial sums.
template <int VEC, int THREADS, typename F>
__device__ __forceinline__ void write_partial(const Pair (&dg)[kPairs], const Pair (&db)[kPairs], int group, int groups,
                                              int lane, int lanes, int cols, F off_of, float* join, float* partial) {
    const int width = lanes * kLaneCols;
    if (group < groups) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float v[kLaneCols];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) (which == 0 ? dg : db)[j].get(v[2 * j], v[2 * j + 1]);
            float* to = join + (group * 2 + which) * width;
#pragma unroll
            for (int k = 0; k < kLaneCols / VEC; ++k) {
                float part[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) part[i] = v[k * VEC + i];
                store_values<float, VEC>(to + (k * lanes + lane) * VEC, VEC, part);
            }
        }
    }
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
        float* out = partial + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * cols;
        for (int c = threadIdx.x; c < cols; c += THREADS) {
            float s = join[which * width + c + off_of(0)];
            for (int g = 1; g < groups; ++g) s += join[(g * 2 + which) * width + c + off_of(g)];
            out[c] = s;
        }
    }
}

// dx of each row, and the block's sums of dy * xh and dy over its rows: each lane adds
// up its own columns, in registers (SHARED: in shared memory, where a block of 1024
// threads has no registers left for them); the groups of a block are joined at the end.
template <typename T, typename W, int VEC, int BLOCK, bool SHARED>
__global__ void __launch_bounds__(BLOCK) norm_backward_kernel(const BackwardArgs<T, W> a) {
    extern __shared__ __align__(16) float join[];
    __shared__ float part[BLOCK / 32][2][2][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lanes = a.lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int groups = BLOCK / lanes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
    GroupSum<2> sum{part[group % (BLOCK / 32)], lanes, 1 + group, 0};
    Pair dg[kPairs], db[kPairs], gamma[kPairs];
    // sum `which` of the lane's element i of its kLaneCols
    const auto mine = [&](int which, int i) -> float& { return join[(which * kLaneCols + i) * lanes + lane]; };
    const auto add_to = [&](int which, int j, Pair v, bool fresh) {
        float lo, hi;
        v.get(lo, hi);
        mine(which, 2 * j) = fresh ? lo : mine(which, 2 * j) + lo;
        mine(which, 2 * j + 1) = fresh ? hi : mine(which, 2 * j + 1) + hi;
    };
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        dg[j] = db[j] = Pair(0.f, 0.f);
        if (SHARED) {
            add_to(0, j, dg[j], true);
            add_to(1, j, db[j], true);
        }
    }
    if (!SHARED) load_weights<W, VEC, kLaneCols>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
    RowPacks<T, VEC, kLaneCols, false> next_x, next_dy;
    float next_mean = 0.f, next_rstd = 0.f;
    const auto ask = [&](int64_t r) {
        next_x.load(a.x + r * a.ldx, lane, lanes, a.cols);
        next_dy.load(a.dy + r * a.lddy, lane, lanes, a.cols);
        next_mean = a.mean[r];
        next_rstd = a.rstd[r];
    };
    if (row < a.rows) ask(row);
    const float inverse_n = 1.f / static_cast<float>(a.cols);
    for (; row < a.rows; row += step) {
        const float mu = next_mean, r = next_rstd;
        Pair hat[kPairs], g[kPairs];
        to_pairs(next_x.p, hat);
        to_pairs(next_dy.p, g);                  // dy: zero past the row's end, as every sum's term there
        if (row + step < a.rows) ask(row + step);
        if (SHARED) load_weights<W, VEC, kLaneCols>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
        const Pair minus(-mu, -mu), r2(r, r);
        Pair sum_g(0.f, 0.f), sum_gx(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            hat[j] = mul2(add2(hat[j], minus), r2);
            if (SHARED) {
                add_to(0, j, mul2(g[j], hat[j]), false);
                add_to(1, j, g[j], false);
            } else {
                dg[j] = fma2(g[j], hat[j], dg[j]);
                db[j] = add2(db[j], g[j]);
            }
            g[j] = mul2(g[j], gamma[j]);
            sum_g = add2(sum_g, g[j]);
            sum_gx = fma2(g[j], hat[j], sum_gx);
        }
        if (!a.dx) continue;
        float s[2];
        row_sums(sum_g, sum_gx, sum, lane, s);
        write_dx<T, VEC, false>(hat, g, s, inverse_n, r2, a.dx + row * a.lddx, lane, lanes, a.cols);
    }
    if (!a.weights) return;
    if (SHARED) {
        __syncthreads();
        copy_partial<VEC, BLOCK>(lanes, a.cols, join, a.partial);
    } else {
        write_partial<VEC, BLOCK>(dg, db, group, groups, lane, lanes, a.cols, [](int) { return 0; }, join, a.partial);
    }
}

// The same through rings of stages that hold a row of x and one of dy.
template <typename T, typename W, int VEC, bool SHIFT>
__global__ void __launch_bounds__(kBackwardRing, 1) norm_backward_ring_kernel(const BackwardArgs<T, W> a, int stages) {
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ RingBarriers barriers;
    __shared__ float part[kBackwardRing / 32][2][2][32];
    const int lanes = a.lanes, groups = kBackwardRing / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    constexpr bool kAny = VEC == 1 || SHIFT;
    const int row_bytes = a.cols * static_cast<int>(sizeof(T)), stage_bytes = ring_stage_bytes(row_bytes, kAny);
    if (threadIdx.x == 0) init_ring(barriers, groups * stages, a.waits);
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    // (threads behind the last whole group have no rows)
    int row = group < groups ? static_cast<int>(blockIdx.x + group * gridDim.x) : static_cast<int>(a.rows);
    Ring<2, kAny> ring{memory + group * stages * 2 * stage_bytes,
                 barriers.full + group * stages,
                 &barriers.waits,
                 a.error,
                 {reinterpret_cast<const uint8_t*>(a.x), reinterpret_cast<const uint8_t*>(a.dy)},
                 {a.ldx * static_cast<int64_t>(sizeof(T)), a.lddy * static_cast<int64_t>(sizeof(T))},
                 static_cast<int>(a.rows),
                 static_cast<int>(groups * gridDim.x),
                 row_bytes,
                 stage_bytes,
                 stages,
                 {0, 0},
                 0};
    if (lane == 0 && group < groups) ring.begin(row);
    const float inverse_n = 1.f / static_cast<float>(a.cols);
    GroupSum<2> sum{part[group], lanes, 1 + group, 0};
    Pair dg[kPairs], db[kPairs], gamma[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dg[j] = db[j] = Pair(0.f, 0.f);
    const int off = SHIFT ? off_of_row(a.x, a.ldx, row) : 0;
    const Span<VEC> span{off, off + a.cols};
    const bool inner = SHIFT && span.holds_all(lane, lanes, kLaneCols / VEC);
    if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int p = (2 * j / VEC * lanes + lane) * VEC + 2 * j % VEC;
            const auto weight = [&](int q) { return !span.has(q) ? 0.f : a.gamma ? to_f32(a.gamma[q - off]) : 1.f; };
            gamma[j] = Pair(weight(p), weight(p + 1));
        }
    } else {
        load_weights<W, VEC, kLaneCols>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
    }
    float next_mean = 0.f, next_rstd = 0.f;
    const auto ask = [&](int64_t r) {
        next_mean = a.mean[r];
        next_rstd = a.rstd[r];
    };
    if (row < ring.rows) ask(row);
    T* dx = a.dx ? a.dx + row * a.lddx : nullptr;
    const int64_t dx_step = a.dx ? ring.step * a.lddx : 0;
    for (; row < ring.rows; row += ring.step, dx += dx_step, ring.turn.next(1, stages)) {
        const float mu = next_mean, r = next_rstd;
        if (row < ring.rows - ring.step) ask(row + ring.step);
        Pair hat[kPairs], g[kPairs];
        {
            RowPacks<T, VEC, kLaneCols, true> x, dy;
            ring.wait();
            const T *from_x = reinterpret_cast<const T*>(ring.at(0, row)), *from_dy = reinterpret_cast<const T*>(ring.at(1, row));
            if (SHIFT && !inner) {
                span.load(x.p, from_x, !ring.direct(row), lane, lanes);
                span.load(dy.p, from_dy, !ring.direct(row), lane, lanes);
            } else {
                x.load(from_x - off, lane, lanes, span.end);
                dy.load(from_dy - off, lane, lanes, span.end);
            }
            to_pairs(x.p, hat);
            to_pairs(dy.p, g);
            if (SHIFT && !inner) {
                span.clear(hat, lane, lanes);
                span.clear(g, lane, lanes);
            }
        }
        const Pair minus(-mu, -mu), r2(r, r);
        Pair sum_g(0.f, 0.f), sum_gx(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            hat[j] = mul2(add2(hat[j], minus), r2);
            dg[j] = fma2(g[j], hat[j], dg[j]);
            db[j] = add2(db[j], g[j]);
            g[j] = mul2(g[j], gamma[j]);
            sum_g = add2(sum_g, g[j]);
            sum_gx = fma2(g[j], hat[j], sum_gx);
        }
        float s[2];
        row_sums(sum_g, sum_gx, sum, lane, s);
        ring.refill(lane, ring.turn.at, row + stages * ring.step);
        if (!a.dx) continue;
        if (SHIFT && !inner) {
            RowPacks<T, VEC, kLaneCols, true> out;
            dx_of(hat, g, s, inverse_n, r2);
            from_pairs(g, out.p);
#pragma unroll
            for (int k = 0; k < kLaneCols / VEC; ++k) span.store(dx, (k * lanes + lane) * VEC, out.p[k]);
        } else {
            write_dx<T, VEC, true>(hat, g, s, inverse_n, r2, dx - off, lane, lanes, span.end);
        }
    }
    if (lane == 0 && group < groups) ring.end();
    if (!a.weights) return;
    __syncthreads();                                     // the rings have been read: their memory joins the groups
    write_partial<VEC, kBackwardRing>(
        dg, db, group, groups, lane, lanes, a.cols,
        [&](int g) { return SHIFT ? off_of_row(a.x, a.ldx, static_cast<int64_t>(blockIdx.x) + g * gridDim.x) : 0; },
        reinterpret_cast<float*>(memory), a.partial);
}

// A lane's columns of a row, in pairs: f(pair, x, dy, gamma).
template <typename T, typename W, int VEC, typename F>
__device__ __forceinline__ void each_pair(const T* x, const T* dy, const Staged<W, VEC>& gamma, int lane, int lanes,
                                          int cols, F f) {
#pragma unroll
    for (int k = 0; k < kLaneCols / VEC; ++k) {
        const int c = (k * lanes + lane) * VEC;
        if (c >= cols) continue;
        const Pack<T, VEC> px = load_pack<T, VEC>(x + c, VEC), pd = load_pack<T, VEC>(dy + c, VEC);
        float g[VEC];
        gamma.get(c, g);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
            f(k * (VEC / 2) + j, pair_of(px, j), pair_of(pd, j), Pair(g[2 * j], g[2 * j + 1]));
    }
}

// The same for rows of more lanes than such a block has (VEC > 1): a block of 1024 threads
// has no registers for a row beside the weight gradients' sums, so the row is read twice from
// its stage, for the sums and for dx, and the stage is refilled when the block has met at the
// next row's barrier.  4096 x 16384 bf16: 193 us with the sums in shared memory, 115 us so (its
// 64 registers a thread spill 28 to 100 bytes); at 8192 columns, where both fit, 110 us against 77.
constexpr int kWideRing = 1024;

template <typename T, typename W, int VEC>
__global__ void __launch_bounds__(kWideRing, 1) norm_backward_wide_ring_kernel(const BackwardArgs<T, W> a, int stages) {
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ RingBarriers barriers;
    __shared__ float part[kWideRing / 32][2][2][32];
    constexpr bool kAny = false;
    const int lanes = a.lanes, groups = 1, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int row_bytes = a.cols * static_cast<int>(sizeof(T)), stage_bytes = ring_stage_bytes(row_bytes, kAny);
    Staged<W, VEC> gamma{reinterpret_cast<W*>(memory + groups * stages * 2 * stage_bytes), lanes * kLaneCols / 2};
    if (threadIdx.x == 0) init_ring(barriers, groups * stages, a.waits);
    __syncthreads();
    wait_for_previous_kernel();
    let_next_kernel_start();
    // (threads behind the last whole group have no rows)
    int row = group < groups ? static_cast<int>(blockIdx.x + group * gridDim.x) : static_cast<int>(a.rows);
    Ring<2, kAny> ring{memory + group * stages * 2 * stage_bytes,
                       barriers.full + group * stages,
                       &barriers.waits,
                       a.error,
                       {reinterpret_cast<const uint8_t*>(a.x), reinterpret_cast<const uint8_t*>(a.dy)},
                       {a.ldx * static_cast<int64_t>(sizeof(T)), a.lddy * static_cast<int64_t>(sizeof(T))},
                       static_cast<int>(a.rows),
                       static_cast<int>(groups * gridDim.x),
                       row_bytes,
                       stage_bytes,
                       stages,
                       {0, 0},
                       0};
    if (lane == 0 && group < groups) ring.begin(row);
    for (int c = threadIdx.x; c < a.cols; c += kWideRing) gamma.put(c, a.gamma ? a.gamma[c] : from_f32<W>(1.f));
    __syncthreads();
    const float inverse_n = 1.f / static_cast<float>(a.cols);
    GroupSum<2> sum{part[group], lanes, 1 + group, 0};
    Pair dg[kPairs], db[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) dg[j] = db[j] = Pair(0.f, 0.f);
    float next_mean = 0.f, next_rstd = 0.f;
    const auto ask = [&](int r) {
        next_mean = a.mean[r];
        next_rstd = a.rstd[r];
    };
    if (row < ring.rows) ask(row);
    int before = -1;                                     // the stage of the group's row before
    for (; row < ring.rows; row += ring.step, ring.turn.next(1, stages)) {
        const float mu = next_mean, r = next_rstd;
        if (row < ring.rows - ring.step) ask(row + ring.step);
        ring.wait();
        const T* const x = reinterpret_cast<const T*>(ring.at(0, row));
        const T* const dy = reinterpret_cast<const T*>(ring.at(1, row));
        const Pair minus(-mu, -mu), r2(r, r);
        Pair sum_g(0.f, 0.f), sum_gx(0.f, 0.f);
        each_pair<T, W, VEC>(x, dy, gamma, lane, lanes, a.cols, [&](int j, Pair v, Pair d, Pair w) {
            const Pair hat = mul2(add2(v, minus), r2), g = mul2(d, w);
            dg[j] = fma2(d, hat, dg[j]);
            db[j] = add2(db[j], d);
            sum_g = add2(sum_g, g);
            sum_gx = fma2(g, hat, sum_gx);
        });
        float s[2];
        row_sums(sum_g, sum_gx, sum, lane, s);
        if (before >= 0) ring.refill(lane, before, row + (stages - 1) * ring.step);
        before = ring.turn.at;
        if (!a.dx) continue;
        // (rstd^2 is not formed: it would leave fp32 before the result does)
        const float mean_g = s[0] * inverse_n, mean_gx = s[1] * inverse_n;
        const Pair minus_g(-mean_g, -mean_g), minus_gx(-mean_gx, -mean_gx);
        T* const dx = a.dx + row * a.lddx;
        Pack<T, VEC> out;
        each_pair<T, W, VEC>(x, dy, gamma, lane, lanes, a.cols, [&](int j, Pair v, Pair d, Pair w) {
            const Pair y = mul2(r2, fma2(d, w, fma2(mul2(add2(v, minus), r2), minus_gx, minus_g)));
            set_pair(out, j % (VEC / 2), y);
            if (j % (VEC / 2) == VEC / 2 - 1) store_pack<T, VEC>(dx + (j / (VEC / 2) * lanes + lane) * VEC, VEC, out);
        });
    }
    if (lane == 0 && group < groups) ring.end();
    if (!a.weights) return;
    __syncthreads();                                     // the rings have been read: their memory joins the groups
    write_partial<VEC, kWideRing>(dg, db, group, groups, lane, lanes, a.cols, [](int) { return 0; }, reinterpret_cast<float*>(memory),
                                  a.partial);
}

// The blocks' sums of 32 columns: eight warps take every eighth block, then join, in an order
// that the sizes alone give.  5 us behind a backward call of 8192 x 8192 (10 MB from L2); sums
// by atomics into dgamma would save it, but their order would change from call to call.
template <typename W>
__global__ void __launch_bounds__(kThreads)
norm_weight_join_kernel(const float* partial, int blocks, int cols, W* dgamma, W* dbeta) {
    __shared__ float part[kThreads / 32][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tiles = (cols + 31) / 32;
    const int which = blockIdx.x / tiles;
    W* out = which == 0 ? dgamma : dbeta;
    if (!out) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x % tiles) * 32 + lane;
    float s = 0.f;
    if (c < cols) {
        constexpr int kAhead = 8;            // loads in flight together: the sums are short chains of them
        const float* at = partial + static_cast<int64_t>(which) * blocks * cols + c;
        for (int b = warp; b < blocks; b += kAhead * (kThreads / 32)) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int row = b + k * (kThreads / 32);
                v[k] = row < blocks ? at[static_cast<int64_t>(row) * cols] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) s += v[k];
        }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    for (int w = 1; w < kThreads / 32; ++w) s += part[w][lane];
    out[c] = from_f32<W>(s);
}

// ---- rows too wide for the registers of a block ------------------------------------
//
// More than 16384 columns.  Each pass reads the row anew (from L2, for rows of some hundred
// KB); plain and right, for widths that hardly any model has (4096 x 20000 bf16: forward 179
// us, 0.27 of the copy bandwidth, backward 430, 0.17).

// The sum over the block, in every thread.
__device__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) v += part[w];
    return v;
}

// One block a row: three passes over the row (sum, squares about the mean, result).
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_forward_wide_kernel(const ForwardArgs<T, W> a) {
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* x = a.x + row * a.ldx;
    T* y = a.y + row * a.ldy;
    float s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) s += to_f32(x[c]);
    const float mu = block_sum(s) / static_cast<float>(a.cols);
    s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const float d = to_f32(x[c]) - mu;
        s += d * d;
    }
    const float r = 1.f / sqrtf(block_sum(s) / static_cast<float>(a.cols) + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const float g = a.gamma ? to_f32(a.gamma[c]) : 1.f, b = a.beta ? to_f32(a.beta[c]) : 0.f;
        y[c] = from_f32<T>((to_f32(x[c]) - mu) * r * g + b);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = r;
    }
}

// One block a row: the row's two sums, then dx.
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_dx_wide_kernel(const BackwardArgs<T, W> a) {
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* x = a.x + row * a.ldx;
    const T* dy = a.dy + row * a.lddy;
    const float mu = a.mean[row], r = a.rstd[row];
    float sg = 0.f, sgx = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const float g = to_f32(dy[c]) * (a.gamma ? to_f32(a.gamma[c]) : 1.f);
        sg += g;
        sgx += g * ((to_f32(x[c]) - mu) * r);
    }
    sg = block_sum(sg) / static_cast<float>(a.cols);
    sgx = block_sum(sgx) / static_cast<float>(a.cols);
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        const float g = to_f32(dy[c]) * (a.gamma ? to_f32(a.gamma[c]) : 1.f);
        a.dx[row * a.lddx + c] = from_f32<T>(r * (g - sg - (to_f32(x[c]) - mu) * r * sgx));
    }
}

// One block per 32 columns: eight warps take every eighth row, then join.
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
norm_weight_grad_wide_kernel(const BackwardArgs<T, W> a, W* dgamma, W* dbeta) {
    __shared__ float part[2][kThreads / 32][32];
    wait_for_previous_kernel();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float dg = 0.f, db = 0.f;
    if (c < a.cols) {
        for (int64_t row = warp; row < a.rows; row += kThreads / 32) {
            const float d = to_f32(a.dy[row * a.lddy + c]);
            dg += d * ((to_f32(a.x[row * a.ldx + c]) - a.mean[row]) * a.rstd[row]);
            db += d;
        }
    }
    part[0][warp][lane] = dg;
    part[1][warp][lane] = db;
    __syncthreads();
    if (warp == 0 && c < a.cols) {
        dg = db = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) {
            dg += part[0][w][lane];
            db += part[1][w][lane];
        }
        if (dgamma) dgamma[c] = from_f32<W>(dg);
        if (dbeta) dbeta[c] = from_f32<W>(db);
    }
}

// ---- launches ----------------------------------------------------------------------

// Lanes of a ring's group: whole warps, `each` columns a lane.
int ring_lanes(int cols, int each) { return ((cols + each - 1) / each + 31) / 32 * 32; }

// Lanes that keep a row of `cols` columns in the register kernels.
int lanes_for(int64_t cols) {
    int lanes = 4;
    while (static_cast<int64_t>(lanes) * kLaneCols < cols) lanes *= 2;
    return lanes;
}

bool in_registers(int64_t cols) { return cols <= static_cast<int64_t>(kMaxLanes) * kLaneCols; }

template <typename T, typename W, int VEC, int BLOCK, bool KEEP>
gemm_status_t forward_rows(const ForwardArgs<T, W>& a, int sms, Queue queue) {
    const int groups = BLOCK / a.lanes;
    const int64_t blocks = (a.rows + groups - 1) / groups;
    const int64_t most = static_cast<int64_t>(sms) * (2048 / BLOCK);
    return launch<norm_forward_kernel<T, W, VEC, BLOCK, KEEP>>(blocks < most ? blocks : most, BLOCK, 0, queue, 1, a);
}

// Stages of a group's ring whose block also needs `fixed` bytes; 0 where rings do not suit:
// rows of no whole packs, rows too short for a copy each (65536 x 256 bf16: 27 us by rings, 23
// in registers; single elements take longer to load, and rings pay from half that length), or
// too few rows.  Forward a quarter of the groups with a row each is enough, as all rows are
// asked for at once (1000 x 4096 bf16 5.3 us, 8.0 in registers; 600 x 4096 4.3 and 5.3; 300 x
// 4096, below the limit, 3.7 and 3.2); backward, with partial sums a block, every group should
// have one (300 x 16384 22 us and 29; 600 x 2048 11.1 and 10.9).
int ring_stages(int cols, int vec, int64_t row_bytes, int sources, int lanes, int threads, int64_t fixed, int64_t rows,
                int sms) {
    const int groups = threads / lanes;
    if (groups == 0 || row_bytes < (vec == 1 ? 512 : 1024) || cols % vec != 0 ||
        rows < int64_t{sms} * groups / (sources == 1 ? 4 : 1) || rows > kRingRows)
        return 0;
    int64_t stages = (kRingShared - fixed) / (row_bytes * sources * groups);
    if (stages > kRingSlots / groups) stages = kRingSlots / groups;
    return stages < 2 ? 0 : static_cast<int>(stages);
}

// Whether rows of both matrices can move in packs off the 16-byte boundaries (see Span), in
// blocks whose rows are multiples of `step` apart.
template <typename T>
bool can_shift(const T* a, int64_t lda, const T* b, int64_t ldb, int64_t step) {
    constexpr int64_t kBytes = sizeof(T);
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0 &&
           (lda - ldb) * kBytes % 16 == 0 && step * lda * kBytes % 16 == 0;
}

// Rows of any length and alignment in packs, through rings; false where that does not suit.
// (fp32 elements are wide enough by themselves: 8000 x 4501 backward 118 us so, 125 in packs;
// and in short rows the warps at the ends are too many: 40000 x 333 fp16 24 and 28 us.)
template <typename T, typename W>
bool forward_shifted(const ForwardArgs<T, W>& a, int sms, Queue queue, gemm_status_t* status) {
    if constexpr (sizeof(T) == 2) {
        constexpr int kCols = 32;
        ForwardArgs<T, W> b = a;
        b.lanes = ring_lanes(a.cols + 7, kCols);
        const int64_t stage = ring_stage_bytes(a.cols * 2, true);
        const int64_t weights = int64_t{2} * b.lanes * kCols * static_cast<int64_t>(sizeof(W));
        const int stages = ring_stages(a.cols, 1, stage, 1, b.lanes, kForwardRing, weights, a.rows, sms);
        if (a.cols <= 512 || stages == 0 || !can_shift<T>(a.x, a.ldx, a.y, a.ldy, sms)) return false;
        const size_t smem = static_cast<size_t>(kForwardRing / b.lanes * stages * stage + weights);
        *status = launch<norm_forward_ring_kernel<T, W, 8, kCols, true>>(sms, kForwardRing, smem, queue, 1, b, stages);
        return true;
    }
    return false;
}

template <typename T, typename W, int VEC>
gemm_status_t forward_vec(const ForwardArgs<T, W>& a, int sms, Queue queue) {
    if constexpr (VEC > 1) {
        // rows that end inside a pack: element by element through rings where there are many
        // that the packs of Span do not take (10000 x 5003 bf16, aligned: 72 us; in registers with
        // a partial pack 141 us)
        const int64_t stage = ring_stage_bytes(a.cols * static_cast<int>(sizeof(T)), true);
        const int lanes = ring_lanes(a.cols, kLaneCols);
        const int64_t weights = int64_t{2} * lanes * kLaneCols * static_cast<int64_t>(sizeof(W));
        if (a.cols % VEC != 0 && ring_stages(a.cols, 1, stage, 1, lanes, kForwardRing, weights, a.rows, sms) > 0)
            return forward_vec<T, W, 1>(a, sms, queue);
    }
    ForwardArgs<T, W> b = a;
    const bool half = VEC > 1 && a.cols > 512;   // 32 columns a lane (single elements take more registers)
    const int each = half ? 32 : 16;
    b.lanes = ring_lanes(a.cols, each);
    const int64_t stage = ring_stage_bytes(a.cols * static_cast<int>(sizeof(T)), VEC == 1);
    const int64_t weights = int64_t{2} * b.lanes * each * static_cast<int64_t>(sizeof(W));
    const int stages = ring_stages(a.cols, VEC, stage, 1, b.lanes, kForwardRing, weights, a.rows, sms);
    if (stages > 0) {
        const size_t smem = static_cast<size_t>(kForwardRing / b.lanes * stages * stage + weights);
        if constexpr (VEC > 1) {
            if (half)
                return launch<norm_forward_ring_kernel<T, W, VEC, 32, false>>(sms, kForwardRing, smem, queue, 1, b, stages);
        }
        return launch<norm_forward_ring_kernel<T, W, VEC, 16, false>>(sms, kForwardRing, smem, queue, 1, b, stages);
    }
    if (a.lanes <= 256) return forward_rows<T, W, VEC, 256, true>(a, sms, queue);
    if (a.lanes == 512) return forward_rows<T, W, VEC, 512, true>(a, sms, queue);
    return forward_rows<T, W, VEC, 1024, false>(a, sms, queue);
}

template <typename T, typename W, int VEC, int BLOCK, bool SHARED>
gemm_status_t backward_rows(const BackwardArgs<T, W>& a, int blocks, Queue queue) {
    // (SHARED keeps its sums there whether they are wanted or not)
    const size_t smem = SHARED || a.weights ? static_cast<size_t>(BLOCK) * kLaneCols * 2 * sizeof(float) : 0;
    return launch<norm_backward_kernel<T, W, VEC, BLOCK, SHARED>>(blocks, BLOCK, smem, queue, 1, a);
}

// Lets the kernels have as much shared memory as their largest launch asks for.
template <typename T, typename W>
gemm_status_t prepare() {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const auto allow = [](auto kernel, int lanes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    lanes * kLaneCols * 2 * static_cast<int>(sizeof(float))) == cudaSuccess;
    };
    const auto allow_ring = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingShared) == cudaSuccess;
    };
    if constexpr (sizeof(T) == 2) {
        if (!allow_ring(norm_forward_ring_kernel<T, W, 8, 32, true>) || !allow_ring(norm_backward_ring_kernel<T, W, 8, true>)) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    if (allow_ring(norm_forward_ring_kernel<T, W, kVec, 16, false>) &&
        allow_ring(norm_forward_ring_kernel<T, W, kVec, 32, false>) &&
        allow_ring(norm_forward_ring_kernel<T, W, 1, 16, false>) &&
        allow_ring(norm_backward_ring_kernel<T, W, kVec, false>) &&
        allow_ring(norm_backward_ring_kernel<T, W, 1, false>) &&
        allow_ring(norm_backward_wide_ring_kernel<T, W, kVec>) &&
        allow(norm_backward_kernel<T, W, kVec, 512, false>, 512) && allow(norm_backward_kernel<T, W, 1, 512, false>, 512) &&
        allow(norm_backward_kernel<T, W, kVec, 1024, true>, 1024) && allow(norm_backward_kernel<T, W, 1, 1024, true>, 1024))
        return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

// Blocks of a backward launch over `rows` rows, and the block size for `lanes`.
int backward_block(int lanes) { return lanes <= 512 ? 512 : 1024; }
int64_t backward_blocks(int64_t rows, int lanes, int sms) {
    const int groups = backward_block(lanes) / lanes;
    const int64_t blocks = (rows + groups - 1) / groups;
    return blocks < sms ? blocks : sms;
}

// Blocks of a ring's backward launch, where the register kernels would have `blocks`: those, or
// as many as give each of the rings' groups two rows (2500 x 125 fp32 13.8 us with the 40 blocks
// of the register kernels' shorter groups).  A block on every SM is not better: a call of 2500 x
// 256 fp32 takes 6.5 us with 79 blocks, beside which the next launch starts, and 9.8 with 152.
int ring_blocks(int64_t rows, int lanes, int blocks, int sms) {
    const int64_t pairs = int64_t{2} * (kBackwardRing / lanes), enough = (rows + pairs - 1) / pairs;
    return enough <= blocks ? blocks : enough < sms ? static_cast<int>(enough) : sms;
}

template <typename T, typename W>
bool backward_shifted(const BackwardArgs<T, W>& a, int* blocks, int sms, Queue queue, gemm_status_t* status) {
    if constexpr (sizeof(T) == 2) {
        BackwardArgs<T, W> b = a;
        b.lanes = ring_lanes(a.cols + 7, kLaneCols);
        const int64_t stage = ring_stage_bytes(a.cols * 2, true);
        const int stages = ring_stages(a.cols, 1, stage, 2, b.lanes, kBackwardRing, 0, a.rows, sms);
        if (stages == 0) return false;
        const int grid = ring_blocks(a.rows, b.lanes, *blocks, sms);
        if (!can_shift<T>(a.x, a.ldx, a.dy, a.lddy, grid) || (a.dx && !can_shift<T>(a.x, a.ldx, a.dx, a.lddx, grid)))
            return false;
        *blocks = grid;
        const int groups = kBackwardRing / b.lanes;
        const size_t ring = static_cast<size_t>(2 * groups * stages * stage);
        const size_t join = static_cast<size_t>(groups * b.lanes) * kLaneCols * 2 * sizeof(float);
        *status = launch<norm_backward_ring_kernel<T, W, 8, true>>(grid, kBackwardRing, ring > join ? ring : join, queue,
                         1, b, stages);
        return true;
    }
    return false;
}

template <typename T, typename W, int VEC>
gemm_status_t backward_vec(const BackwardArgs<T, W>& a, int* blocks, int sms, Queue queue) {
    BackwardArgs<T, W> b = a;
    b.lanes = ring_lanes(a.cols, kLaneCols);
    const int64_t stage = ring_stage_bytes(a.cols * static_cast<int>(sizeof(T)), VEC == 1);
    const int stages = ring_stages(a.cols, VEC, stage, 2, b.lanes, kBackwardRing, 0, a.rows, sms);
    if (stages > 0) {
        const size_t ring = static_cast<size_t>(2 * (kBackwardRing / b.lanes) * stages * stage);
        const size_t join = static_cast<size_t>(kBackwardRing / b.lanes * b.lanes) * kLaneCols * 2 * sizeof(float);
        *blocks = ring_blocks(a.rows, b.lanes, *blocks, sms);
        return launch<norm_backward_ring_kernel<T, W, VEC, false>>(*blocks, kBackwardRing, ring > join ? ring : join, queue, 1,
                      b, stages);
    }
    if constexpr (VEC > 1) {
        const int64_t weights = static_cast<int64_t>(b.lanes) * kLaneCols * static_cast<int64_t>(sizeof(W));
        const int wide = b.lanes > kBackwardRing ? ring_stages(a.cols, VEC, stage, 2, b.lanes, kWideRing, weights, a.rows, sms) : 0;
        const size_t ring = static_cast<size_t>(2 * wide * stage + weights);
        const size_t join = static_cast<size_t>(b.lanes) * kLaneCols * 2 * sizeof(float);
        if (wide > 0)
            return launch<norm_backward_wide_ring_kernel<T, W, VEC>>(*blocks, kWideRing, ring > join ? ring : join, queue, 1,
                                                                     b, wide);
    }
    if (a.lanes <= 512) return backward_rows<T, W, VEC, 512, false>(a, *blocks, queue);
    return backward_rows<T, W, VEC, 1024, true>(a, *blocks, queue);
}

// Calls f with values of the plan's element and weight types.
template <typename F>
gemm_status_t with_types(const gemm_norm_plan* p, F f) {
    return with_elem(p->elem, [&](auto t) {
        if (p->weight_elem == GEMM_ELEM_F32) return f(t, float());
        return f(t, t);
    });
}

}  // namespace
}  // namespace gbt

extern "C" {

gemm_status_t gemm_norm_plan_create(int64_t max_rows, int64_t cols, gemm_elem_t elem,
                                    gemm_elem_t weight_elem, gemm_norm_plan_t* plan) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!gbt::valid_elem(elem) || (weight_elem != elem && weight_elem != GEMM_ELEM_F32))
        return GEMM_ERR_UNSUPPORTED;
    if (max_rows < 0 || max_rows > INT32_MAX || cols < 1 || cols > gbt::kMostColumns)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    const gemm_status_t st = gbt::begin_plan(&device, &sms);
    if (st != GEMM_OK) return st;
    size_t sums = 0;
    if (max_rows > 0 && gbt::in_registers(cols)) {
        // (rings take no fewer rows than SMs, and have no more blocks)
        const int64_t blocks = max_rows >= sms ? sms : gbt::backward_blocks(max_rows, gbt::lanes_for(cols), sms);
        sums = static_cast<size_t>(blocks * cols) * 2 * sizeof(float);
    }
    void* memory = nullptr;
    gemm_status_t room = gbt::allocate(&memory, 256 + sums);
    if (room != GEMM_OK) return room;
    gemm_norm_plan* p = new (std::nothrow) gemm_norm_plan();
    if (!p || gbt::clear_now(memory, 256) != GEMM_OK) {
        cudaFree(memory);
        room = p ? GEMM_ERR_CUDA : GEMM_ERR_OOM;
        delete p;
        return room;
    }
    p->max_rows = max_rows;
    p->cols = cols;
    p->elem = elem;
    p->weight_elem = weight_elem;
    p->device = device;
    p->num_sms = sms;
    p->memory = memory;
    p->error_word = static_cast<int32_t*>(memory);
    p->partial = reinterpret_cast<float*>(static_cast<uint8_t*>(memory) + 256);
    const gemm_status_t ready =
        gbt::with_types(p, [](auto t, auto v) { return gbt::prepare<decltype(t), decltype(v)>(); });
    if (ready != GEMM_OK) {
        cudaFree(memory);
        delete p;
        return ready;
    }
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_norm_forward(gemm_norm_plan_t p, int64_t rows, const void* x, int64_t ldx,
                                const void* gamma, const void* beta, float eps, void* y,
                                int64_t ldy, float* mean, float* rstd, void* stream) {
    if (!p || rows < 0 || rows > p->max_rows || !(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y || ldx < p->cols || ldy < p->cols)) return GEMM_ERR_INVALID_ARG;
    const int e = gbt::elem_bytes(p->elem), w = gbt::elem_bytes(p->weight_elem);
    if (!gbt::aligned(x, e) || !gbt::aligned(y, e) || !gbt::aligned(gamma, w) ||
        !gbt::aligned(beta, w) || !gbt::aligned(mean, 4) || !gbt::aligned(rstd, 4))
        return GEMM_ERR_ALIGNMENT;
    const gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK || rows == 0) return st;
    const gbt::Queue queue{stream, p->device};
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        const gbt::ForwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const W*>(gamma),
                                       static_cast<const W*>(beta), static_cast<T*>(y), mean, rstd,
                                       p->error_word, ldx, ldy, rows, eps, static_cast<int>(p->cols),
                                       gbt::lanes_for(p->cols), p->waits};
        if (!gbt::in_registers(p->cols))
            return gbt::launch<gbt::norm_forward_wide_kernel<T, W>>(rows, gbt::kThreads, 0, queue, 1, a);
        const bool vec = gbt::rows_aligned(x, ldx, e) && gbt::rows_aligned(y, ldy, e) &&
                         gbt::aligned(gamma, 16) && gbt::aligned(beta, 16);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        const bool whole = vec && p->cols % kVec == 0;
        gemm_status_t status = GEMM_OK;
        if (!whole && gbt::forward_shifted<T, W>(a, p->num_sms, queue, &status)) return status;
        return vec ? gbt::forward_vec<T, W, kVec>(a, p->num_sms, queue)
                   : gbt::forward_vec<T, W, 1>(a, p->num_sms, queue);
    });
}

gemm_status_t gemm_norm_backward(gemm_norm_plan_t p, int64_t rows, const void* x, int64_t ldx,
                                 const void* gamma, const float* mean, const float* rstd,
                                 const void* dy, int64_t lddy, void* dx, int64_t lddx,
                                 void* dgamma, void* dbeta, void* stream) {
    if (!p || rows < 0 || rows > p->max_rows) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !dy || !mean || !rstd || ldx < p->cols || lddy < p->cols ||
                     (dx && lddx < p->cols)))
        return GEMM_ERR_INVALID_ARG;
    const int e = gbt::elem_bytes(p->elem), w = gbt::elem_bytes(p->weight_elem);
    if (!gbt::aligned(x, e) || !gbt::aligned(dy, e) || !gbt::aligned(dx, e) ||
        !gbt::aligned(gamma, w) || !gbt::aligned(dgamma, w) || !gbt::aligned(dbeta, w) ||
        !gbt::aligned(mean, 4) || !gbt::aligned(rstd, 4))
        return GEMM_ERR_ALIGNMENT;
    gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK) return st;
    const gbt::Queue queue{stream, p->device};
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        W* dg = static_cast<W*>(dgamma);
        W* db = static_cast<W*>(dbeta);
        const int lanes = gbt::lanes_for(p->cols);
        gbt::BackwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const W*>(gamma), mean, rstd,
                                  static_cast<const T*>(dy), static_cast<T*>(dx), p->partial, p->error_word, ldx,
                                  lddy, lddx, rows, static_cast<int>(p->cols), lanes, dg || db, p->waits};
        const int tiles = static_cast<int>((p->cols + 31) / 32);
        gemm_status_t s = GEMM_OK;
        if (!gbt::in_registers(p->cols)) {
            // (the weight's gradients first: dx may overwrite dy or x)
            if (a.weights)
                s = gbt::launch<gbt::norm_weight_grad_wide_kernel<T, W>>(tiles, gbt::kThreads, 0, queue,
                                1, a, dg, db);
            if (s == GEMM_OK && dx && rows > 0)
                s = gbt::launch<gbt::norm_dx_wide_kernel<T, W>>(rows, gbt::kThreads, 0, queue, 1, a);
            return s;
        }
        int blocks = static_cast<int>(gbt::backward_blocks(rows, lanes, p->num_sms));
        if (blocks > 0) {
            const bool vec = gbt::rows_aligned(x, ldx, e) && gbt::rows_aligned(dy, lddy, e) &&
                             (!dx || gbt::rows_aligned(dx, lddx, e)) && gbt::aligned(gamma, 16);
            constexpr int kVec = 16 / static_cast<int>(sizeof(T));
            const bool whole = vec && p->cols % kVec == 0;
            if (whole || !gbt::backward_shifted<T, W>(a, &blocks, p->num_sms, queue, &s))
                s = vec ? gbt::backward_vec<T, W, kVec>(a, &blocks, p->num_sms, queue)
                        : gbt::backward_vec<T, W, 1>(a, &blocks, p->num_sms, queue);
        }
        if (s == GEMM_OK && a.weights)
            s = gbt::launch<gbt::norm_weight_join_kernel<W>>(2 * tiles, gbt::kThreads, 0, queue, 1,
                            p->partial, blocks, static_cast<int>(p->cols), dg, db);
        return s;
    });
}

gemm_status_t gemm_norm_plan_set_timeout(gemm_norm_plan_t p, uint64_t ns) {
    return p ? gbt::set_wait_limit(&p->waits, ns) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_norm_plan_set_wait_test(gemm_norm_plan_t p, uint32_t extra_bytes, uint32_t every) {
    return p ? gbt::set_wait_test(&p->waits, extra_bytes, every) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_norm_plan_check(gemm_norm_plan_t p, void* stream) {
    return p ? gbt::check_error_word(p->error_word, stream) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_norm_plan_destroy(gemm_norm_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->memory) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
