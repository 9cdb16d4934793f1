// train_distill.cu -- the distillation loss of gemm_train.h against a teacher's top
// logits, forward and backward.
#include <float.h>
#include <math.h>

#include <new>

#include "train_common.cuh"

namespace gbt {
// How the pipeline over rows cuts a row and fills the GPU (see distill_stream_kernel).
struct StreamShape {
    int pieces, piece, stages, slots;
    int clusters;            // resident at once; 0 = not used
    size_t smem;
};
}  // namespace gbt

struct gemm_distill_plan {
    int64_t max_rows, vocab, max_top;
    gemm_elem_t elem;
    int device, num_sms;
    int32_t* error_word;
    float2* sums;            // of rows that no cluster can hold: maximum and sum, between the directions
    gbt::Waits waits;
    gbt::StreamShape forward, both;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 1024;
constexpr int kMaxCluster = 8;                 // blocks that share a row
constexpr int kPieceBytes = 32 * 1024;         // of a row that a block aims to hold
constexpr int kMostPieceBytes = 200 * 1024;    // ... and can hold
constexpr int kMostShared = 224 * 1024;        // dynamic shared memory of any launch
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Mode { kForward = 1, kBackward = 2, kBoth = 3 };

struct Teacher {
    const void* ids;
    const void* values;
    const float* lse;
    int64_t ld_ids, ld_values;
    int top, id_type, value_elem;
};

template <typename T>
struct Args {
    const T* logits;
    T* dlogits;
    const float* dloss;
    float* loss;
    float* lse;
    int32_t* error;
    float2* sums;          // each row's maximum and sum, where both directions are two kernels
    Teacher teacher;
    int64_t ldl, ldd;
    float temperature, inverse, c;      // ... one over it, log2(e) over it
    int vocab, piece;      // elements; a piece is a multiple of the pack
    int pieces;            // of a row: blocks that share it
    Waits waits;
};

// ---- asynchronous copies ----------------------------------------------------------

// The elements of [src, src + n) into shared memory at dst, which has src's offset
// from a 16-byte boundary: one thread starts a bulk copy of the whole 16-byte units
// (counted on the barrier), all threads copy the ragged ends.  Past the ends, up to
// the 16-byte boundaries, go -infinities.  `extra`: see Waits.
template <typename T>
__device__ __forceinline__ void start_copy(T* dst, const T* src, int n, uint64_t* barrier, uint32_t extra) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
    int head = (VEC - off) % VEC;                    // elements before the first boundary
    if (head > n) head = n;
    const int body = (n - head) / VEC * VEC, tail = n - head - body;
    if (threadIdx.x == 0) {
        const uint32_t bytes = static_cast<uint32_t>(body * static_cast<int>(sizeof(T)));
        expect_bytes(barrier, bytes + extra);
        if (bytes > 0) copy_bytes(dst + head, src + head, bytes, barrier);
    }
    if (threadIdx.x < VEC) {
        const int i = threadIdx.x;
        if (i < head) dst[i] = src[i];
        if (i < tail) dst[head + body + i] = src[head + body + i];
        if (i < off) dst[i - off] = from_f32<T>(-INFINITY);
        const int end = off + n, fill = (VEC - end % VEC) % VEC;
        if (i < fill) dst[n + i] = from_f32<T>(-INFINITY);
    }
}

// ---- the teacher's entries ----------------------------------------------------------

// In shared memory, `top` each: ids (-1 = no entry), log2 of the probabilities, the
// probabilities.
struct Entries {
    int32_t* id;
    float* log2p;
    float* p;
    float* x;      // the student's logits at the ids (where a kernel fetches them)
    float* own;    // sum of p over an id's equals at its first entry, -1 at the others
};

// One warp: a row's entries; returns the mass.  Values are scaled to log2 units by
// c = log2(e) / temperature.  `logits`: the row's, whose values at the ids go to en.x, or
// null.  The loads of kBatch * 32 entries are in flight together.
template <typename T>
__device__ float load_entries(const Entries& en, const Teacher& t, int64_t row, const T* logits, float c,
                              int vocab, int32_t* error) {
    constexpr int kBatch = 4;
    const int lane = threadIdx.x % 32;
    const float given = t.lse ? t.lse[row] * kLog2e : 0.f;
    float high = -INFINITY, sum = 0.f;
    for (int j0 = lane; j0 < t.top; j0 += 32 * kBatch) {
        int64_t id[kBatch];
        float v[kBatch], x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u * 32;
            id[u] = j < t.top ? load_index(t.ids, row * t.ld_ids + j, t.id_type) : -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u * 32;
            v[u] = j < t.top ? load_elem(t.values, row * t.ld_values + j, t.value_elem) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (id[u] >= vocab) {
                atomicOr(error, kErrorIndex);
                id[u] = -1;
            }
            x[u] = logits && id[u] >= 0 ? to_f32(logits[id[u]]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int j = j0 + u * 32;
            if (j >= t.top) break;
            const float own = id[u] < 0 ? -INFINITY : v[u];
            en.id[j] = id[u] < 0 ? -1 : static_cast<int32_t>(id[u]);
            en.log2p[j] = own;
            if (logits) en.x[j] = x[u];
            high = fmaxf(high, own);
        }
    }
    // log2 p = (v - base) c - rest: the largest value is taken off before the values are scaled
    float base = 0.f, rest = given;
    if (!t.lse) {
        high = warp_max(high);
        base = high == -INFINITY ? 0.f : high;
        for (int j = lane; j < t.top; j += 32) sum += exp2_fast((en.log2p[j] - base) * c);
        rest = log2f(warp_sum(sum));
    }
    sum = 0.f;
    for (int j = lane; j < t.top; j += 32) {
        const float l = en.log2p[j] == -INFINITY ? -INFINITY : fmaf(en.log2p[j] - base, c, -rest);
        en.log2p[j] = l;
        en.p[j] = exp2_fast(l);
        sum += en.p[j];
    }
    return warp_sum(sum);
}

// Asks L2 for a row's entries.
__device__ void prefetch_entries(const Teacher& t, int64_t row) {
    const auto ask = [](const void* p, int64_t offset, int bytes) {
        for (int b = threadIdx.x % 32 * 128; b < bytes; b += 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" :: "l"(static_cast<const uint8_t*>(p) + offset + b));
    };
    const int id_bytes = t.id_type == GEMM_INDEX_I64 ? 8 : 4, value_bytes = t.value_elem == GEMM_ELEM_F32 ? 4 : 2;
    ask(t.ids, row * t.ld_ids * id_bytes, t.top * id_bytes);
    ask(t.values, row * t.ld_values * value_bytes, t.top * value_bytes);
}

// One warp, after load_entries: fills `own`.  Ids are compared four at a time; equal
// ones are rare.
__device__ void join_equal_ids(const Entries& en, int top) {
    __syncwarp();
    for (int j = threadIdx.x % 32; j < top; j += 32) {
        const int id = en.id[j];
        float p = en.p[j];
        if (id >= 0) {
            bool equal = false;
            for (int k = 0; k < top; k += 4) {
                const int4 v = *reinterpret_cast<const int4*>(en.id + k);   // (16-byte aligned)
                equal = equal || (v.x == id && k != j) || (v.y == id && k + 1 != j && k + 1 < top) ||
                        (v.z == id && k + 2 != j && k + 2 < top) || (v.w == id && k + 3 != j && k + 3 < top);
            }
            if (equal) {
                bool leads = true;
                p = 0.f;
                for (int k = 0; k < top; ++k) {
                    if (en.id[k] != id) continue;
                    p += en.p[k];
                    leads = leads && k >= j;
                }
                if (!leads) p = -1.f;
            }
        }
        en.own[j] = id >= 0 ? p : -1.f;
    }
}

// ---- running maximum and sum ----------------------------------------------------------
//
// One pass over the row gives both.  Of a set of logits s: m = max s and sum exp2((s - m) c), c
// being log2(e) / temperature.  Where |m c| is below kNear, that is exp2(s c - k) with k = m c
// rounded, one instruction for two logits, times exp2 of that rounding, which is exact and
// applied once.  Further out it would be exp2 of hundreds: there the maximum is subtracted
// from the logits first.  (Without that, rows at masks of -1e10 gave infinities or nothing.)
// A maximum below the limit of masks (-infinity, or a type's lowest value) is that of masked
// logits only: their sum counts from zero and is zero.

constexpr float kMasked = -1e30f * kLog2e;    // m c, of a logit of -1e30 times the temperature
constexpr float kNear = 268435456.f;          // 2^28: m c is rounded by 16 at most
constexpr float kNearGiven = 4194304.f;       // 2^22: a given log-sum-exp, by a fifth

__device__ __forceinline__ float finite_base(float m, float c) { return m * c < kMasked ? 0.f : m; }

// Of a set of logits and teacher entries: m, the sum, the entries' part of the loss, p (log2 p -
// (x - m) c), x being the logit at the entry, and their mass.
struct alignas(16) Part {
    float m, sum, terms, here;
    // The same, counted from a maximum that is no lower.
    __device__ __forceinline__ void count_from(float high, float c) {
        const float d = (m - finite_base(high, c)) * c;
        sum *= exp2_fast(d);
        if (here != 0.f) terms -= here * d;
        m = high;
    }
    __device__ __forceinline__ void add_entry(float p, float log2p, float x, float c) {
        if (x > m) count_from(x, c);
        terms += p * (log2p - (x - finite_base(m, c)) * c);
        here += p;
    }
};

// The parts of LANES neighbouring lanes joined, in each of them (ENTRIES: with terms and mass).
template <int LANES, bool ENTRIES>
__device__ __forceinline__ void join_lanes(Part& p, float c) {
    float high = p.m;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
    p.count_from(high, c);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        p.sum += __shfl_xor_sync(0xffffffffu, p.sum, o);
        if (ENTRIES) {
            p.terms += __shfl_xor_sync(0xffffffffu, p.terms, o);
            p.here += __shfl_xor_sync(0xffffffffu, p.here, o);
        }
    }
}

// The parts of a row's blocks joined, by a whole warp.
__device__ __forceinline__ Part join_blocks(const Part* parts, int blocks, float c) {
    if (blocks == 2) {
        Part all = parts[0], other = parts[1];
        const float high = fmaxf(all.m, other.m);
        all.count_from(high, c);
        other.count_from(high, c);
        all.sum += other.sum;
        all.terms += other.terms;
        all.here += other.here;
        return all;
    }
    const int r = threadIdx.x % kMaxCluster;
    Part all = r < blocks ? parts[r] : Part{-INFINITY, 0.f, 0.f, 0.f};
    join_lanes<kMaxCluster, true>(all, c);
    return all;
}

// The sum over a thread's packs of a row (first, first + step, ... of those from the 16-byte
// boundary off elements before src on) counted from their maximum m.  It is rare; the pipeline
// over fp32 rows takes 9% longer with it inside, short rows 4% longer with a call.
template <typename T>
__device__ __forceinline__ float far_sum(const T* src, int off, int n, int first, int step, float m, float c) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const float base = finite_base(m, c);
    float sum = 0.f;
#pragma unroll 1
    for (int at = first * VEC - off; at < n; at += step * VEC)
#pragma unroll 1
        for (int i = 0; i < VEC; ++i)
            if (at + i >= 0 && at + i < n) sum += exp2_fast((to_f32(src[at + i]) - base) * c);
    return sum;
}
template <typename T>
__device__ __noinline__ float call_far_sum(const T* src, int off, int n, int first, int step, float m, float c) {
    return far_sum(src, off, n, first, step, m, c);
}

template <typename T>
struct Running {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    float m = -INFINITY, k = -INFINITY;       // the maximum, and that times c
    Pair sum = Pair(0.f, 0.f), sum_b = Pair(0.f, 0.f);

    // (below -kNear the sum counts from zero and is zero)
    template <int N>
    __device__ __forceinline__ void add(const Pack<T, VEC> (&q)[N], float c) {
        m = fmaxf(m, pack_max(q));
        const float high = m * c, base = high < -kNear ? 0.f : high;
        const float shrink = exp2_fast(k - base);
        k = high;
        sum = mul2(sum, Pair(shrink, shrink));
        sum_b = mul2(sum_b, Pair(shrink, shrink));
        const Pair c2(c, c), base2(-base, -base);
#pragma unroll
        for (int b = 0; b < N; ++b) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                float lo, hi;
                fma2(pair_of(q[b], j), c2, base2).get(lo, hi);
                Pair& to = j & 1 ? sum_b : sum;
                to = add2(to, Pair(exp2_fast(lo), exp2_fast(hi)));
            }
        }
    }
    // The logits' part; far from zero they are read once more (see far_sum).
    __device__ __forceinline__ Part total(float c, const T* src, int off, int n, int first, int step) const {
        float lo, hi;
        add2(sum, sum_b).get(lo, hi);
        lo += hi;
        if (fabsf(k) < kNear) return Part{m, lo * exp2_fast(-fmaf(m, c, -k)), 0.f, 0.f};
        if (k < kMasked) return Part{m, lo, 0.f, 0.f};
        return Part{m, call_far_sum(src, off, n, first, step, m, c), 0.f, 0.f};
    }
};

// The smaller of the number and zero; NaN stays.
__device__ __forceinline__ float at_most_zero(float v) {
    asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(v));
    return v;
}

// A row's softmax, from a forward pass' maximum and sum, between which nothing is rounded, or
// from a given log-sum-exp.  Near: q = inverse * exp2(s c - k), inverse making up for the
// rounding of k.  Far: q = inverse * exp2((s - base) c + rest), at most inverse (a given
// log-sum-exp has the rounding of its own size, which is large there).
struct Softmax {
    float base, k, rest, inverse;
    bool far;
    __device__ __forceinline__ void of_sum(const Part& row, float c) {
        base = finite_base(row.m, c);
        k = base * c;
        far = !(fabsf(k) < kNear);
        rest = 0.f;
        inverse = __fdividef(far ? 1.f : exp2_fast(-fmaf(base, c, -k)), row.sum);
    }
    // (far, whatever the size)
    __device__ __forceinline__ void of_sum_over(const Part& row, float c) {
        *this = Softmax{finite_base(row.m, c), 0.f, 0.f, __fdividef(1.f, row.sum), true};
    }
    __device__ __forceinline__ void of_lse(float lse, float temperature, float c) {
        base = lse * temperature;
        k = base * c;
        far = !(fabsf(k) < kNearGiven);
        rest = fmaf(-lse, temperature, base) * c;
        inverse = far ? 1.f : exp2_fast(rest - fmaf(base, c, -k));
    }
    // q over inverse, at a logit
    __device__ __forceinline__ float at(float s, float c) const {
        return exp2_fast(far ? at_most_zero(fmaf(s - base, c, rest)) : fmaf(s, c, -k));
    }
    // the log-sum-exp, from the forward pass' sum
    __device__ __forceinline__ float lse(float sum, float inverse_temperature) const {
        return fmaf(base, inverse_temperature, kLn2 * log2f(sum));
    }
};

// exp2((s - base) c) of two logits: what short rows take whatever their size (a second path for
// far rows cost 4% of their time, this one instruction nothing).
__device__ __forceinline__ Pair exp2_over(Pair s, Pair minus_base, Pair c) {
    float lo, hi;
    mul2(add2(s, minus_base), c).get(lo, hi);
    return Pair(exp2_fast(lo), exp2_fast(hi));
}

// The sum of that over some packs.
template <typename T, int VEC, int N>
__device__ __forceinline__ float sum_over(const Pack<T, VEC> (&q)[N], float base, float c) {
    const Pair c2(c, c), base2(-base, -base);
    Pair sum(0.f, 0.f), sum_b(0.f, 0.f);
#pragma unroll
    for (int b = 0; b < N; ++b) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            Pair& to = j & 1 ? sum_b : sum;
            to = add2(to, exp2_over(pair_of(q[b], j), base2, c2));
        }
    }
    float lo, hi;
    add2(sum, sum_b).get(lo, hi);
    return lo + hi;
}

template <typename T>
__device__ __forceinline__ Pack<T, 16 / sizeof(T)> all_masked() {
    Pack<T, 16 / static_cast<int>(sizeof(T))> q;
#pragma unroll
    for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i) q.set(i, -INFINITY);
    return q;
}

// scale * exp2(s c - k) of each element of a pack.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> gradient(const Pack<T, VEC>& q, float c, float k, float scale) {
    Pack<T, VEC> g;
    const Pair c2(c, c), all2(-k, -k), scale2(scale, scale);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        float lo, hi;
        fma2(pair_of(q, j), c2, all2).get(lo, hi);
        set_pair(g, j, mul2(scale2, Pair(exp2_fast(lo), exp2_fast(hi))));
    }
    return g;
}

// The same by exp2_over.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> gradient_over(const Pack<T, VEC>& q, float c, float base, float scale) {
    Pack<T, VEC> g;
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j)
        set_pair(g, j, mul2(Pair(scale, scale), exp2_over(pair_of(q, j), Pair(-base, -base), Pair(c, c))));
    return g;
}

// ---- the kernel ------------------------------------------------------------------------
//
// A block holds one piece of a row's logits in shared memory.  Forward: the blocks of a
// row form a cluster; each finds its piece's maximum and sum in one pass, and they
// exchange those and their parts of the loss.  Backward: the gradient of the piece, from the
// piece.  Both: the piece is read from memory once.
//
// Serves calls of few rows, whose pieces fill the GPU (33 x 32000 fp32, forward: 4.4 us, the
// chain of load, sum and exchange), and every backward call but those of short rows: there
// blocks are independent and six or more an SM hide one another's waits (2048 x 50021 fp16: 62
// us, 0.96 of the copy bandwidth; 67 with six blocks an SM for 16-bit logits instead of eight).
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, MODE != kBackward ? 4 : sizeof(T) == 2 ? 8 : 6) distill_kernel(const Args<T> a) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    constexpr bool kLoss = (MODE & kForward) != 0, kGrad = (MODE & kBackward) != 0;
    extern __shared__ __align__(16) uint8_t memory[];
    __shared__ uint64_t barrier;
    __shared__ Part exchange[kMaxCluster];
    __shared__ Part part[kWarps];
    __shared__ float row_mass;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t row = blockIdx.x / static_cast<unsigned>(a.pieces);
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.pieces));
    const int top = a.teacher.top;
    const bool shared_row = kLoss && a.pieces > 1;
    Entries en;
    en.id = reinterpret_cast<int32_t*>(memory);
    en.log2p = reinterpret_cast<float*>(en.id + top);
    en.p = en.log2p + top;
    // behind the entries, one pack of room before and after the piece
    T* const room = reinterpret_cast<T*>(memory + (top * 12 + 15) / 16 * 16);
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(shared_address(&barrier)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (shared_row) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    wait_for_previous_kernel();
    let_next_kernel_start();

    const float c = a.c;
    if (warp == 0) {
        const float mass = load_entries<T>(en, a.teacher, row, nullptr, c, a.vocab, a.error);
        if (lane == 0) row_mass = mass;
    }
    float given_lse = 0.f;
    if (MODE == kBackward) given_lse = a.lse[row];
    __syncthreads();
    const float mass = row_mass;
    const bool out = mass == 0.f || (MODE == kBackward && given_lse == -INFINITY);
    const int begin = rank * a.piece;
    const int n = min(a.piece, a.vocab - begin);         // (at least one: pieces are not empty)
    T* d = nullptr;
    if (kGrad) d = a.dlogits + row * a.ldd + begin;

    Softmax row_q = {0.f, 0.f, 0.f, 0.f, false};
    if (MODE == kBackward && !out) {
        if (a.sums) {
            const float2 row_sum = a.sums[row];
            row_q.of_sum({row_sum.x, row_sum.y, 0.f, 0.f}, c);
        } else {
            row_q.of_lse(given_lse, a.temperature, c);
        }
    }
    bool empty = out;
    const T* src = a.logits + row * a.ldl + begin;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
    T* const s = room + off;
    const int packs = (off + n + VEC - 1) / VEC;         // from room on
    bool arrived = true;
    if (!out) {
        start_copy(s, src, n, &barrier, a.waits.extra_bytes());
        arrived = wait_phase(&barrier, 0, a.waits.limit);
        if (!arrived) atomicOr(a.error, kErrorTimeout);
        __syncthreads();                                 // the ragged ends
    }
    if (kLoss) {
        Running<T> run;
        if (!out) {
            constexpr int kBatch = 2;
            for (int at = tid; at < packs; at += kBatch * kThreads) {
                Pack<T, VEC> q[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    q[b] = at + b * kThreads < packs ? load_pack<T, VEC>(room + (at + b * kThreads) * VEC, VEC)
                                                     : all_masked<T>();
                run.add(q, c);
            }
        }
        Part mine = run.total(c, s, off, n, tid, kThreads);
        join_lanes<32, false>(mine, c);
        if (lane == 0) part[warp] = mine;
        __syncthreads();
        // the piece's, and the entries in it
        if (warp == 0) {
            mine = part[lane % kWarps];
            join_lanes<kWarps, false>(mine, c);
            if (!out) {
                const float base = finite_base(mine.m, c);
                for (int j = lane; j < top; j += 32) {
                    const int at = en.id[j] - begin;
                    if (en.id[j] >= 0 && at >= 0 && at < n && !(en.p[j] == 0.f)) {
                        mine.terms += en.p[j] * (en.log2p[j] - (to_f32(s[at]) - base) * c);
                        mine.here += en.p[j];
                    }
                }
                mine.terms = warp_sum(mine.terms);
                mine.here = warp_sum(mine.here);
            }
            if (shared_row) {
                __syncwarp();
                // every block has started: put this block's numbers into each one's memory
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (lane < a.pieces) {
                    uint32_t remote;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(remote) : "r"(shared_address(&exchange[rank])), "r"(lane));
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(remote), "f"(mine.m), "f"(mine.sum), "f"(mine.terms), "f"(mine.here)
                                 : "memory");
                }
            } else if (lane == 0) {
                exchange[0] = mine;
            }
        } else if (shared_row) {
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
        if (shared_row) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
        const Part all = join_blocks(exchange, a.pieces, c);
        row_q.of_sum(all, c);
        empty = out || all.sum == 0.f;
        if (rank == 0 && tid == 0) {
            const float total = all.terms + mass * log2f(all.sum);
            a.loss[row] = empty ? 0.f : a.temperature * a.temperature * kLn2 * total;
            a.lse[row] = empty ? -INFINITY : row_q.lse(all.sum, a.inverse);
        }
    }
    if (!kGrad) {
        if (!arrived) wait_phase(&barrier, 0, a.waits.limit);   // no copy may land in a finished block's memory
        return;
    }

    const bool same = (reinterpret_cast<uintptr_t>(d) & 15u) == (reinterpret_cast<uintptr_t>(src) & 15u);
    const float scale = a.temperature * (a.dloss ? a.dloss[row] : 1.f);
    const float q_scale = scale * (mass * row_q.inverse);
    if (!empty && row_q.far) {
#pragma unroll 1
        for (int i = tid; i < n; i += kThreads) d[i] = from_f32<T>(q_scale * row_q.at(to_f32(s[i]), c));
    } else for (int k = tid; k < packs; k += kThreads) {
        Pack<T, VEC> g;
        if (empty) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) g.set(i, 0.f);
        } else {
            g = gradient(load_pack<T, VEC>(room + k * VEC, VEC), c, row_q.k, q_scale);
        }
        const int at = k * VEC - off;                    // the pack's first element in the piece
        if (same && at >= 0 && at + VEC <= n) {
            store_pack<T, VEC>(d + at, VEC, g);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (at + i >= 0 && at + i < n) d[at + i] = reinterpret_cast<const T*>(&g.raw)[i];
        }
    }
    if (!empty) {
        __syncthreads();                                 // the stores above come first
        for (int j = tid; j < top; j += kThreads) {
            const int id = en.id[j], at = id - begin;
            if (id < 0 || at < 0 || at >= n) continue;
            float p = 0.f;
            bool first = true;                           // of equal ids the first writes for all
            for (int k = 0; k < top; ++k) {
                if (en.id[k] != id) continue;
                p += en.p[k];
                first = first && k >= j;
            }
            if (first)
                d[at] = from_f32<T>(scale * (mass * row_q.inverse * row_q.at(to_f32(s[at]), c) - p));
        }
    }
    if (!arrived) wait_phase(&barrier, 0, a.waits.limit);       // (as above)
}

// ---- many rows: a pipeline over rows -----------------------------------------------------
//
// A block (or a cluster, each block with its part of the row) goes through rows, with
// three kinds of warps: one copies the logits into a ring of stages, as far ahead as there
// is room; some prepare the teacher's entries of the next rows (each is a chain of loads,
// which take some microseconds behind the copies); the others compute.  Forward frees a
// stage as soon as it is summed; both directions together keep the row's stages until its
// gradient is written, and copy the next row into those that are free.  So memory is busy
// while a row is reduced, and no block starts or ends per row.
//
// Bound by bytes.  Forward, 4096 x 128000 bf16, top 64: 154 us, 0.96 of the copy bandwidth
// (with unpaired arithmetic 209, and 384 then by a block per piece of a row).  Both directions,
// 4096 x 64000 bf16: 167 us, 0.91; parts of at most 64 KB and two blocks an SM, so that one
// block's stores go beside the other's sums (three blocks of 32-KB parts 171).  Three warps for
// the entries, 16-KB stages and logits at the ids taken from the ring were 169 where one warp,
// 8-KB stages and loads of those logits were 201.  With 200 entries a row, 387 us: the search
// for equal ids, 200 x 200 a row by one warp, is what takes them.  Forward pays from few rows
// on: 455 rows of 128000, the last count before this kernel, take 42 us by the one above,
// 456 take 22; both directions 151 and 152 rows of 64000, 15 us each.
//
// When a wait runs out (the block's patience is over, and no later wait lasts), nothing more is
// copied, prepared or exchanged, and the computing warps go on through their rows with whatever
// there is (leaving the loop cost 3% of the time).  So how many barriers a row has depends on no
// data, and what a warp does together on nothing that its lanes may see differently.  Before
// the block ends, what it asked for and what the other blocks of its cluster sent it lands, by
// count.

template <int MODE> constexpr int kStageBytesOf = MODE == kBoth ? 16384 : 8192;
constexpr int kMostStages = 16;
constexpr int kEntryWords = 5;     // arrays of Entries
constexpr int kComputeWarps = 8;
constexpr int kComputeThreads = kComputeWarps * 32;
constexpr int kEntryWarps = 3;     // each prepares every third row's entries
constexpr int kMostSlots = 2 * kEntryWarps;
constexpr int kFirstCompute = 32 * (1 + kEntryWarps);
constexpr int kStreamThreads = kFirstCompute + kComputeThreads;

struct StreamBarriers {
    uint64_t full[kMostStages], empty[kMostStages];
    uint64_t entries_full[kMostSlots], entries_empty[kMostSlots];
    uint64_t exchanged[2];
    Part exchange[2][kMaxCluster];
    Part part[2][kComputeWarps];
    float mass[kMostSlots], scale[kMostSlots];
    uint32_t sent[kMaxCluster];      // exchanges that each block of the cluster took part in, at its end
    uint32_t patience;       // ns that a wait may last; 0: one ran out, nothing waits any more
    uint32_t extra;          // bytes that a stage waits for beyond its copies (see Waits)
};

__device__ __forceinline__ void compute_barrier() {
    asm volatile("bar.sync 1, %0;" :: "n"(kComputeThreads) : "memory");
}

// The block's warps meet once more, each kind at the end of its part.
__device__ __forceinline__ void end_of_block() {
    __syncwarp();
    asm volatile("bar.sync 0;" ::: "memory");
}

// Takes bytes that will not come off what the barrier's phase waits for.
__device__ __forceinline__ void strike_bytes(uint64_t* barrier, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.shared::cta.b64 [%0], %1;" :: "r"(shared_address(barrier)), "r"(bytes) : "memory");
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kStreamThreads, MODE == kBoth ? 2 : 3)
distill_stream_kernel(const Args<T> a, int64_t rows, int stages, int slots) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    constexpr int kStageBytes = kStageBytesOf<MODE>;
    constexpr int kStage = kStageBytes / static_cast<int>(sizeof(T));     // elements
    constexpr bool kGrad = MODE == kBoth;
    constexpr bool kSplit = kGrad;               // a row may be a cluster's (else a.pieces is 1)
    constexpr int kBatch = kStage / VEC / kComputeThreads;                // packs a thread takes of a stage
    extern __shared__ __align__(16) uint8_t memory[];
    __shared__ StreamBarriers sh;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const unsigned pieces = kSplit ? static_cast<unsigned>(a.pieces) : 1u;
    const int rank = static_cast<int>(blockIdx.x % pieces);
    const int64_t first = blockIdx.x / pieces;
    const int64_t step = gridDim.x / pieces;
    const int top = a.teacher.top;
    const int padded_top = (top + 3) / 4 * 4;
    T* const ring = reinterpret_cast<T*>(memory);
    const auto entries = [&](int slot) {
        float* at = reinterpret_cast<float*>(memory + stages * kStageBytes) + slot * kEntryWords * padded_top;
        return Entries{reinterpret_cast<int32_t*>(at), at + padded_top, at + 2 * padded_top, at + 3 * padded_top,
                       at + 4 * padded_top};
    };
    const int begin = rank * a.piece;
    const int n = min(a.piece, a.vocab - begin);
    // (divided here and below, not on the host as for the other kernels: 900 x 128000 fp32 both
    // directions took 165 us with that, 149 so, in whatever way it changes the order of things)
    const float c = kLog2e / a.temperature;
    if (tid == 0) {
        for (int k = 0; k < stages; ++k) {
            init_barrier(&sh.full[k], 1);
            init_barrier(&sh.empty[k], kComputeWarps);
        }
        for (int k = 0; k < slots; ++k) {
            init_barrier(&sh.entries_full[k], 1);
            init_barrier(&sh.entries_empty[k], kComputeWarps + 1);
        }
        for (int k = 0; k < 2; ++k) init_barrier(&sh.exchanged[k], 1);
        sh.patience = a.waits.limit;
        sh.extra = a.waits.extra_bytes();
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (kSplit && a.pieces > 1) cluster_barrier();       // the others' barriers exist
    wait_for_previous_kernel();
    let_next_kernel_start();

    uint32_t sent = 0, received = 0;                     // exchanges that the first computing warp took part in and saw whole
    if (warp == 0) {                                     // copies
        Turn stage{0, 0}, turn{0, 0};
        uint32_t issued = 0;                             // (lane 0)
        for (int64_t row = first; row < rows; row += step, turn.next(1, slots)) {
            const int slot = turn.at;
            wait_or_die(&sh.entries_full[slot], turn.round & 1, &sh.patience, a.error);
            const bool out = __shfl_sync(0xffffffffu, sh.mass[slot], 0) == 0.f;
            if (lane == 0) arrive(&sh.entries_empty[slot]);
            if (out) continue;
            const T* src = a.logits + row * a.ldl + begin;
            const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
            const T* base = src - off;                   // the 16-byte boundary at or before src
            const int end = off + n;                     // positions count from there
            const int head_end = min((off + VEC - 1) / VEC * VEC, end);
            const int tail_begin = max(end / VEC * VEC, head_end);
            T head = from_f32<T>(-INFINITY), tail = head;
            if (lane < VEC) {                            // the ragged ends, by plain loads
                if (off > 0 && lane >= off && lane < head_end) head = base[lane];
                if (tail_begin + lane < end) tail = base[tail_begin + lane];
            }
            for (int at = 0; at < end; at += kStage) {
                wait_or_die(&sh.empty[stage.at], (stage.round & 1) ^ 1, &sh.patience, a.error);
                T* const to = ring + stage.at * kStage;
                const int lo = at == 0 ? head_end : at, hi = min(at + kStage, tail_begin);
                const bool first_pack = at == 0 && off > 0;
                const bool last_pack = tail_begin < end && tail_begin >= at && tail_begin < at + kStage;
                if (first_pack || last_pack) {
                    if (first_pack && lane < VEC) to[lane] = head;
                    if (last_pack && lane < VEC) to[tail_begin - at + lane] = tail;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                // (a warp that gave up has left its stages unread: they are not filled again)
                if (lane == 0 && !is_dead(&sh.patience)) {
                    const uint32_t bytes = hi > lo ? static_cast<uint32_t>((hi - lo) * static_cast<int>(sizeof(T))) : 0;
                    expect_bytes(&sh.full[stage.at], bytes + sh.extra);
                    if (bytes > 0) copy_bytes(to + (lo - at), base + lo, bytes, &sh.full[stage.at]);
                    ++issued;
                }
                stage.next(1, stages);
            }
        }
        end_of_block();
        // A wait that ran out may have left copies behind: let them land (bounded).
        if (lane == 0 && is_dead(&sh.patience)) {
            const uint32_t began = timer_ns(), n_stages = static_cast<uint32_t>(stages);
            for (uint32_t k = issued > n_stages ? issued - n_stages : 0; k < issued; ++k)
                wait_until(&sh.full[k % n_stages], k / n_stages & 1, began, a.waits.limit);
        }
        __syncwarp();
    } else if (warp <= kEntryWarps) {                    // the teacher's entries
        Turn turn{warp - 1, 0};
        for (int64_t row = first + (warp - 1) * step; row < rows;
             row += kEntryWarps * step, turn.next(kEntryWarps, slots)) {
            const int slot = turn.at;
            if (!__all_sync(0xffffffffu, wait_or_die(&sh.entries_empty[slot], (turn.round & 1) ^ 1, &sh.patience, a.error)))
                break;
            const Entries en = entries(slot);
            if (row + kEntryWarps * step < rows) prefetch_entries(a.teacher, row + kEntryWarps * step);
            const float dloss = kGrad && a.dloss ? a.dloss[row] : 1.f;
            const float mass = load_entries<T>(en, a.teacher, row, kGrad ? nullptr : a.logits + row * a.ldl, c,
                                              a.vocab, a.error);
            if (kGrad) join_equal_ids(en, top);
            if (lane == 0) {
                sh.mass[slot] = mass;
                if (kGrad) sh.scale[slot] = a.temperature * dloss;
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.entries_full[slot]);
        }
        end_of_block();
    } else {                                             // the arithmetic
        const int thread = tid - kFirstCompute, worker = warp - kFirstCompute / 32;
        Turn stage{0, 0}, entry{0, 0};
        uint32_t exchanges = 0;
        for (int64_t row = first; row < rows; row += step, entry.next(1, slots)) {
            const int slot = entry.at;
            wait_or_die(&sh.entries_full[slot], entry.round & 1, &sh.patience, a.error);
            const float mass = __shfl_sync(0xffffffffu, sh.mass[slot], 0);
            const Entries en = entries(slot);
            const bool out = mass == 0.f;
            const T* src = a.logits + row * a.ldl + begin;
            const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
            const int packs = (off + n + VEC - 1) / VEC;
            const Turn row_stage = stage;
            bool empty = out;
            Softmax row_q = {0.f, 0.f, 0.f, 0.f, false};
            Part all = {0.f, 0.f, 0.f, 0.f};
            if (out) {
                compute_barrier();
            } else {
                Running<T> run;
                for (int p0 = 0; p0 < packs; p0 += kStage / VEC) {
                    wait_or_die(&sh.full[stage.at], stage.round & 1, &sh.patience, a.error);
                    const T* from = ring + stage.at * kStage + thread * VEC;
                    Pack<T, VEC> q[kBatch];
                    if (packs - p0 >= kStage / VEC) {
#pragma unroll
                        for (int b = 0; b < kBatch; ++b) q[b] = load_pack<T, VEC>(from + b * kComputeThreads * VEC, VEC);
                    } else {
#pragma unroll
                        for (int b = 0; b < kBatch; ++b)
                            q[b] = p0 + thread + b * kComputeThreads < packs
                                       ? load_pack<T, VEC>(from + b * kComputeThreads * VEC, VEC)
                                       : all_masked<T>();
                    }
                    if (!kGrad) {
                        __syncwarp();
                        if (lane == 0) arrive(&sh.empty[stage.at]);
                    }
                    run.add(q, c);
                    stage.next(1, stages);
                }
                // and the entries of this part
                all = run.total(c, src, off, n, thread, kComputeThreads);        // (the stages may have gone)
                for (int j = thread; j < top; j += kComputeThreads) {
                    const int at = en.id[j] - begin;
                    if (en.id[j] < 0 || at < 0 || at >= n) continue;
                    if (kGrad) {                         // the row's stages still hold its logits
                        int s = row_stage.at + (off + at) / kStage;
                        if (s >= stages) s -= stages;
                        en.x[j] = to_f32(ring[s * kStage + (off + at) % kStage]);
                    }
                    if (!(en.p[j] == 0.f)) all.add_entry(en.p[j], en.log2p[j], en.x[j], c);
                }
                join_lanes<32, true>(all, c);
                const int turn = exchanges & 1;
                if (lane == 0) sh.part[turn][worker] = all;
                compute_barrier();
                all = sh.part[turn][lane % kComputeWarps];
                join_lanes<kComputeWarps, true>(all, c);
                if (kSplit && a.pieces > 1) {
                    // this block's numbers, to each block of the row (none any more once a wait has run out)
                    if (worker == 0 && __shfl_sync(0xffffffffu, is_dead(&sh.patience), 0) == 0) {
                        if (lane == 0)
                            expect_bytes(&sh.exchanged[turn], static_cast<uint32_t>(a.pieces) * 16);
                        if (lane < a.pieces) {
                            uint32_t slot_at, barrier_at;
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                         : "=r"(slot_at) : "r"(shared_address(&sh.exchange[turn][rank])), "r"(lane));
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                         : "=r"(barrier_at) : "r"(shared_address(&sh.exchanged[turn])), "r"(lane));
                            asm volatile(
                                "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
                                "[%5];"
                                :: "r"(slot_at), "f"(all.m), "f"(all.sum), "f"(all.terms), "f"(all.here), "r"(barrier_at) : "memory");
                        }
                        ++sent;
                        __syncwarp();
                    }
                    if (wait_or_die(&sh.exchanged[turn], (exchanges >> 1) & 1, &sh.patience, a.error) && sent > exchanges)
                        received = sent;
                    all = join_blocks(sh.exchange[turn], a.pieces, c);
                }
                ++exchanges;
                empty = all.sum == 0.f;
                row_q.of_sum(all, c);
            }
            if (rank == 0 && thread == 0) {
                const float total = all.terms + mass * log2f(all.sum);
                a.loss[row] = empty ? 0.f : a.temperature * a.temperature * kLn2 * total;
                a.lse[row] = empty ? -INFINITY : row_q.lse(all.sum, 1.f / a.temperature);
            }
            if (kGrad) {
                T* const d = a.dlogits + row * a.ldd + begin;
                const bool same = (reinterpret_cast<uintptr_t>(d) & 15u) == (reinterpret_cast<uintptr_t>(src) & 15u);
                const float scale = sh.scale[slot];
                const float q_scale = scale * (mass * row_q.inverse);
                stage = row_stage;
                if (!empty && row_q.far) {
#pragma unroll 1
                    for (int i = thread; i < n; i += kComputeThreads) {
                        int s = row_stage.at + (off + i) / kStage;
                        if (s >= stages) s -= stages;
                        d[i] = from_f32<T>(q_scale * row_q.at(to_f32(ring[s * kStage + (off + i) % kStage]), c));
                    }
                    __syncwarp();
                    for (int p0 = 0; p0 < packs; p0 += kStage / VEC) {
                        if (lane == 0) arrive(&sh.empty[stage.at]);
                        stage.next(1, stages);
                    }
                } else for (int p0 = 0; p0 < packs; p0 += kStage / VEC) {
                    const T* from = ring + stage.at * kStage;
                    const int at0 = (p0 + thread) * VEC - off;       // of the first pack, in the piece
                    if (!empty && same && p0 * VEC >= off && p0 * VEC - off + kStage <= n) {
#pragma unroll
                        for (int b = 0; b < kBatch; ++b)
                            store_pack<T, VEC>(d + at0 + b * kComputeThreads * VEC, VEC,
                                               gradient(load_pack<T, VEC>(from + (thread + b * kComputeThreads) * VEC, VEC),
                                                        c, row_q.k, q_scale));
                    } else {
                        for (int b = 0; b < kBatch; ++b) {
                            const int mine = thread + b * kComputeThreads, at = at0 + b * kComputeThreads * VEC;
                            if (p0 + mine >= packs) break;
                            Pack<T, VEC> g;
                            if (empty) {
#pragma unroll
                                for (int i = 0; i < VEC; ++i) g.set(i, 0.f);
                            } else {
                                g = gradient(load_pack<T, VEC>(from + mine * VEC, VEC), c, row_q.k, q_scale);
                            }
                            if (same && at >= 0 && at + VEC <= n) {
                                store_pack<T, VEC>(d + at, VEC, g);
                            } else {
#pragma unroll
                                for (int i = 0; i < VEC; ++i)
                                    if (at + i >= 0 && at + i < n) d[at + i] = reinterpret_cast<const T*>(&g.raw)[i];
                            }
                        }
                    }
                    if (!out) {
                        __syncwarp();
                        if (lane == 0) arrive(&sh.empty[stage.at]);
                        stage.next(1, stages);
                    }
                }
                compute_barrier();                       // the stores above come first
                if (!empty) {
                    for (int j = thread; j < top; j += kComputeThreads) {
                        const float p = en.own[j];
                        const int at = en.id[j] - begin;
                        if (p >= 0.f && at >= 0 && at < n)
                            d[at] = from_f32<T>(scale * (mass * row_q.inverse * row_q.at(en.x[j], c) - p));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&sh.entries_empty[slot]);
        }
        if (kSplit && a.pieces > 1 && worker == 0 && lane < a.pieces) {
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(remote) : "r"(shared_address(&sh.sent[rank])), "r"(lane));
            asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(remote), "r"(sent) : "memory");
        }
        end_of_block();
    }
    if (!kSplit || a.pieces == 1) return;
    cluster_barrier();                                   // no block leaves while others write to it
    if (tid == kFirstCompute) {
        // ... and none while their numbers are on the way: those that were sent and not waited for.
        const uint32_t began = timer_ns();
        for (uint32_t e = received;; ++e) {
            uint32_t coming = 0;
            for (int r = 0; r < a.pieces; ++r) coming += sh.sent[r] > e ? 1 : 0;
            if (e >= sent && coming == 0) break;
            const uint32_t missing = static_cast<uint32_t>(a.pieces) - coming;
            if (e >= sent)
                expect_bytes(&sh.exchanged[e & 1], coming * 16);
            else if (missing > 0)                        // (all were expected)
                strike_bytes(&sh.exchanged[e & 1], missing * 16);
            wait_until(&sh.exchanged[e & 1], (e >> 1) & 1, began, a.waits.limit);
        }
    }
}

// ---- short rows ---------------------------------------------------------------------------
//
// A warp keeps a whole row in registers, PACKS packs a lane, and asks for it before it
// prepares the teacher's entries.  No block-wide step: for rows of some hundred logits the
// blocks' and barriers' time of the other kernels is several times that of the memory (16384
// x 1000 bf16, both directions, 16 entries a row: 24 us, 64 entries 36).  Bound by the entries' chain of loads and sums, which is
// most of the work of such a row (16384 x 250, 16 entries:
// 18 us).
// Blocks an SM that are worth holding the registers down for (none spills but the
// 16-bit forward kernels of 8 packs, 32 bytes): 16384 x 1000 bf16 both directions 24 us, 29 with
// a block less.
template <typename T, int MODE, int PACKS>
constexpr int kShortBlocks = sizeof(T) == 4 ? (PACKS == 2 ? 5 : PACKS == 4 ? 4 : PACKS == 8 ? 3 : 2)
                             : MODE == kForward ? (PACKS <= 4 ? 5 : PACKS == 8 ? 4 : 2)
                             : PACKS == 2 ? 5 : PACKS == 4 ? 4 : MODE == kBackward ? (PACKS == 8 ? 3 : 2) : PACKS == 8 ? 2 : 1;

template <typename T, int MODE, int PACKS>
__global__ void __launch_bounds__(kThreads, kShortBlocks<T, MODE, PACKS>) distill_short_kernel(const Args<T> a, int64_t rows) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    constexpr bool kLoss = (MODE & kForward) != 0, kGrad = (MODE & kBackward) != 0;
    extern __shared__ __align__(16) uint8_t memory[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int top = a.teacher.top, padded_top = (top + 3) / 4 * 4, n = a.vocab;
    float* const mine = reinterpret_cast<float*>(memory) + warp * kEntryWords * padded_top;
    const Entries en{reinterpret_cast<int32_t*>(mine), mine + padded_top, mine + 2 * padded_top,
                     mine + 3 * padded_top, mine + 4 * padded_top};
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (row >= rows) return;
    const T* src = a.logits + row * a.ldl;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
    Pack<T, VEC> q[PACKS];
#pragma unroll
    for (int b = 0; b < PACKS; ++b) {
        const int at = (b * 32 + lane) * VEC - off;      // the pack's first element in the row
        if (at >= 0 && at + VEC <= n) {
            q[b] = load_pack<T, VEC>(src + at, VEC);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                q[b].set_raw(i, at + i >= 0 && at + i < n ? src[at + i] : from_f32<T>(-INFINITY));
        }
    }
    const float given = MODE == kBackward ? a.lse[row] : 0.f;
    const float scale = kGrad ? a.temperature * (a.dloss ? a.dloss[row] : 1.f) : 0.f;
    const float c = a.c;
    const float mass = load_entries(en, a.teacher, row, src, c, n, a.error);
    if (kGrad) join_equal_ids(en, top);
    bool empty = mass == 0.f || (MODE == kBackward && given == -INFINITY);
    Softmax row_q = {0.f, 0.f, 0.f, 0.f, false};
    if (MODE == kBackward) row_q.of_lse(given, a.temperature, c);
    if (kLoss) {
        Part all = {warp_max(pack_max(q)), 0.f, 0.f, 0.f};
        all.sum = warp_sum(sum_over(q, finite_base(all.m, c), c));
        empty = empty || all.sum == 0.f;
        row_q.of_sum_over(all, c);
        if (!empty)
            for (int j = lane; j < top; j += 32)
                if (!(en.p[j] == 0.f)) all.terms += en.p[j] * (en.log2p[j] - (en.x[j] - row_q.base) * c);
        all.terms = warp_sum(all.terms);
        if (lane == 0) {
            a.loss[row] = empty ? 0.f : a.temperature * a.temperature * kLn2 * (all.terms + mass * log2f(all.sum));
            a.lse[row] = empty ? -INFINITY : row_q.lse(all.sum, a.inverse);
        }
    }
    if (!kGrad) return;
    T* const d = a.dlogits + row * a.ldd;
    const bool same = (reinterpret_cast<uintptr_t>(d) & 15u) == (reinterpret_cast<uintptr_t>(src) & 15u);
    const float q_scale = empty ? 0.f : scale * (mass * row_q.inverse);
    __syncwarp();                                        // the row has been read: d may be the logits
    if (MODE == kBackward && !empty && row_q.far) {
#pragma unroll 1
        for (int i = lane; i < n; i += 32) d[i] = from_f32<T>(q_scale * row_q.at(to_f32(src[i]), c));
    } else
#pragma unroll
    for (int b = 0; b < PACKS; ++b) {
        const int at = (b * 32 + lane) * VEC - off;
        Pack<T, VEC> g;
        if (empty) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) g.set(i, 0.f);
        } else {
            g = kLoss ? gradient_over(q[b], c, row_q.base, q_scale) : gradient(q[b], c, row_q.k, q_scale);
        }
        if (same && at >= 0 && at + VEC <= n) {
            store_pack<T, VEC>(d + at, VEC, g);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (at + i >= 0 && at + i < n) d[at + i] = reinterpret_cast<const T*>(&g.raw)[i];
        }
    }
    if (empty) return;
    __syncwarp();                                        // the stores above come first
    for (int j = lane; j < top; j += 32)
        if (en.own[j] >= 0.f)
            d[en.id[j]] =
                from_f32<T>(scale * (mass * row_q.inverse * row_q.at(en.x[j], c) - en.own[j]));
}

// ---- rows that no cluster can hold ---------------------------------------------------------

// Forward over few rows that no cluster can hold (more than 1.6 MB each; many such rows go
// through the pipeline): one block a row, a pass for the maximum and one for the sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) distill_forward_wide_kernel(const Args<T> a) {
    extern __shared__ __align__(16) uint8_t memory[];
    __shared__ Part part[kWarps];
    __shared__ float row_mass;
    const int top = a.teacher.top, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Entries en;
    en.id = reinterpret_cast<int32_t*>(memory);
    en.log2p = reinterpret_cast<float*>(en.id + top);
    en.p = en.log2p + top;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t row = blockIdx.x;
    const T* s = a.logits + row * a.ldl;
    const float c = a.c;
    if (warp == 0) {
        const float mass = load_entries<T>(en, a.teacher, row, nullptr, c, a.vocab, a.error);
        if (lane == 0) row_mass = mass;
    }
    __syncthreads();
    const float mass = row_mass;
    Part all = {-INFINITY, 0.f, 0.f, 0.f};
    if (mass != 0.f) {
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) all.m = fmaxf(all.m, to_f32(s[i]));
        const float base = finite_base(all.m, c);
        for (int i = threadIdx.x; i < a.vocab; i += kThreads) all.sum += exp2_fast((to_f32(s[i]) - base) * c);
    }
    join_lanes<32, false>(all, c);
    if (lane == 0) part[warp] = all;
    __syncthreads();
    if (warp != 0) return;
    all = part[lane % kWarps];
    join_lanes<kWarps, false>(all, c);
    const bool empty = mass == 0.f || all.sum == 0.f;
    Softmax row_q;
    row_q.of_sum(all, c);
    if (a.sums && lane == 0) a.sums[row] = make_float2(all.m, all.sum);
    if (!empty)
        for (int j = lane; j < top; j += 32)
            if (!(en.p[j] == 0.f)) all.terms += en.p[j] * (en.log2p[j] - (to_f32(s[en.id[j]]) - row_q.base) * c);
    all.terms = warp_sum(all.terms);
    if (lane == 0) {
        a.loss[row] = empty ? 0.f : a.temperature * a.temperature * kLn2 * (all.terms + mass * log2f(all.sum));
        a.lse[row] = empty ? -INFINITY : row_q.lse(all.sum, a.inverse);
    }
}

// How a row is cut: pieces of about kPieceBytes, more and smaller ones where there are
// too few rows to fill the GPU, at most `most`.
template <typename T>
void cut_row(Args<T>& a, int64_t rows, int sms, int64_t most) {
    constexpr int64_t kVec = 16 / sizeof(T);
    const int64_t bytes = static_cast<int64_t>(a.vocab) * static_cast<int64_t>(sizeof(T));
    int64_t pieces = 1;
    while (pieces < most && bytes > pieces * kPieceBytes) pieces *= 2;
    while (pieces < most && pieces < kMaxCluster && rows * pieces < 2 * sms && bytes > pieces * 8192) pieces *= 2;
    const int64_t packs = (a.vocab + kVec - 1) / kVec;
    const int64_t each = (packs + pieces - 1) / pieces;
    a.piece = static_cast<int>(each * kVec);
    a.pieces = static_cast<int>((packs + each - 1) / each);
}

// Rows that a warp's registers hold: up to 16 packs a lane, wherever the row begins.
template <typename T>
bool is_short(int64_t vocab) {
    return vocab + 16 / static_cast<int>(sizeof(T)) - 1 <= 16 * 32 * (16 / static_cast<int>(sizeof(T)));
}

template <typename T, int MODE>
gemm_status_t run_short(const Args<T>& a, int64_t rows, Queue queue) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const int lanes = (a.vocab + VEC - 1 + VEC - 1) / VEC;        // packs of a row, wherever it begins
    const int64_t blocks = (rows + kWarps - 1) / kWarps;
    const size_t smem = kWarps * kEntryWords * sizeof(float) * ((a.teacher.top + 3) / 4 * 4);
    if (lanes <= 2 * 32) return launch<distill_short_kernel<T, MODE, 2>>(blocks, kThreads, smem, queue, 1, a, rows);
    if (lanes <= 4 * 32) return launch<distill_short_kernel<T, MODE, 4>>(blocks, kThreads, smem, queue, 1, a, rows);
    if (lanes <= 8 * 32) return launch<distill_short_kernel<T, MODE, 8>>(blocks, kThreads, smem, queue, 1, a, rows);
    return launch<distill_short_kernel<T, MODE, 16>>(blocks, kThreads, smem, queue, 1, a, rows);
}

template <typename T, int MODE>
gemm_status_t run(Args<T> a, int64_t rows, int sms, Queue queue) {
    if (is_short<T>(a.vocab)) return run_short<T, MODE>(a, rows, queue);
    cut_row(a, rows, sms, MODE == kBackward ? INT32_MAX : kMaxCluster);
    const size_t smem = (a.teacher.top * 12 + 15) / 16 * 16 + a.piece * sizeof(T) + 32;
    return launch<distill_kernel<T, MODE>>(rows * a.pieces, kThreads, smem, queue,
                  MODE == kBackward ? 1 : a.pieces, a);
}

// Lets the kernels have as much shared memory as the largest launch asks for.
template <typename T, int MODE>
bool prepare_short() {
    const int most = kWarps * kEntryWords * static_cast<int>(sizeof(float)) * kMaxTop;
    const auto allow = [&](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess;
    };
    return allow(distill_short_kernel<T, MODE, 2>) && allow(distill_short_kernel<T, MODE, 4>) &&
           allow(distill_short_kernel<T, MODE, 8>) && allow(distill_short_kernel<T, MODE, 16>);
}

template <typename T>
gemm_status_t prepare() {
    const auto allow = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) == cudaSuccess;
    };
    if (prepare_short<T, kForward>() && prepare_short<T, kBackward>() && prepare_short<T, kBoth>() &&
        allow(distill_stream_kernel<T, kForward>) && allow(distill_stream_kernel<T, kBoth>) &&
        allow(distill_kernel<T, kForward>) && allow(distill_kernel<T, kBackward>) && allow(distill_kernel<T, kBoth>))
        return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

template <typename T, int MODE>
gemm_status_t run_stream(Args<T> a, const StreamShape& shape, int64_t rows, Queue queue) {
    a.piece = shape.piece;
    a.pieces = shape.pieces;
    const int64_t clusters = rows < shape.clusters ? rows : shape.clusters;
    return launch<distill_stream_kernel<T, MODE>>(clusters * a.pieces, kStreamThreads, shape.smem, queue,
                  a.pieces, a, rows, shape.stages, shape.slots);
}

// The pipeline's shape for a plan; clusters == 0 where it does not suit.
template <typename T, int MODE>
StreamShape stream_shape(int64_t vocab, int64_t max_top) {
    constexpr int64_t kVec = 16 / sizeof(T);
    constexpr int64_t kStageBytes = kStageBytesOf<MODE>;
    const int64_t bytes = vocab * static_cast<int64_t>(sizeof(T));
    StreamShape shape = {};
    if (is_short<T>(vocab)) return shape;
    const int64_t slot = kEntryWords * sizeof(float) * ((max_top + 3) / 4 * 4);
    shape.slots = slot * kMostSlots <= 16 * 1024 ? kMostSlots : kEntryWarps;
    const int64_t entries = slot * shape.slots;
    const int64_t room = (kMostShared - entries) / kStageBytes;
    shape.pieces = 1;
    int64_t stages = 6;
    if (MODE == kBoth) {
        while (shape.pieces < kMaxCluster && bytes > shape.pieces * int64_t{64 * 1024}) shape.pieces *= 2;
        const int64_t packs = (vocab + kVec - 1) / kVec;
        const int64_t each = (packs + shape.pieces - 1) / shape.pieces;
        shape.piece = static_cast<int>(each * kVec);
        shape.pieces = static_cast<int>((packs + each - 1) / each);
        const int64_t need = ((each + 1) * 16 + kStageBytes - 1) / kStageBytes;
        stages = need <= 2 ? 4 : need <= 4 ? 6 : 13;
        if (stages > room) stages = room;
        if (need > stages) return shape;
    } else {
        shape.piece = static_cast<int>(vocab);
    }
    shape.stages = static_cast<int>(stages);
    shape.smem = static_cast<size_t>(stages * kStageBytes + entries);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(shape.pieces * 1024));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = shape.smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(shape.pieces);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&shape.clusters, distill_stream_kernel<T, MODE>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        shape.clusters = 0;
    }
    return shape;
}

template <typename T>
gemm_status_t run_forward_wide(const Args<T>& a, int64_t rows, Queue queue) {
    return launch<distill_forward_wide_kernel<T>>(rows, kThreads, a.teacher.top * 12, queue, 1, a);
}

// Whether a cluster can hold a row.
bool fits(int64_t vocab, int bytes) { return vocab * bytes <= int64_t{kMaxCluster} * kMostPieceBytes; }

gemm_status_t check_call(const gemm_distill_plan* p, int64_t rows, const void* logits, int64_t ldl,
                         const gemm_teacher_t* t, float temperature) {
    if (!p || rows < 0 || rows > p->max_rows || !t) return GEMM_ERR_INVALID_ARG;
    if (!valid_index(t->id_type) || !valid_elem(t->value_elem)) return GEMM_ERR_UNSUPPORTED;
    // (a normal number: of others the scale, or the product with a masked logit, is none)
    if (!(temperature >= FLT_MIN && temperature <= FLT_MAX) || t->top < 0 || t->top > p->max_top) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!logits || ldl < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && t->top > 0 &&
        (!t->ids || !t->values || t->ld_ids < t->top || t->ld_values < t->top))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned(logits, elem_bytes(p->elem)) || !aligned(t->ids, index_bytes(t->id_type)) ||
        !aligned(t->values, elem_bytes(t->value_elem)) || !aligned(t->lse, 4))
        return GEMM_ERR_ALIGNMENT;
    return check_device(p->device);
}

template <typename T>
Args<T> arguments(const gemm_distill_plan* p, const void* logits, int64_t ldl, const gemm_teacher_t* t,
                  float temperature) {
    Args<T> a = {};
    a.logits = static_cast<const T*>(logits);
    a.ldl = ldl;
    a.teacher = Teacher{t->ids,
                        t->values,
                        t->lse,
                        t->ld_ids,
                        t->ld_values,
                        static_cast<int>(t->top),
                        static_cast<int>(t->id_type),
                        static_cast<int>(t->value_elem)};
    a.temperature = temperature;
    a.inverse = 1.f / temperature;
    a.c = kLog2e / temperature;
    a.vocab = static_cast<int>(p->vocab);
    a.error = p->error_word;
    a.waits = p->waits;
    return a;
}

}  // namespace
}  // namespace gbt

extern "C" {

gemm_status_t gemm_distill_plan_create(int64_t max_rows, int64_t vocab, int64_t max_top,
                                       gemm_elem_t elem, gemm_distill_plan_t* plan) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!gbt::valid_elem(elem)) return GEMM_ERR_UNSUPPORTED;
    if (max_rows < 0 || max_rows > INT32_MAX || vocab < 1 || vocab > gbt::kMostColumns || max_top < 0 ||
        max_top > gbt::kMaxTop)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    gemm_status_t st = gbt::begin_plan(&device, &sms);
    if (st != GEMM_OK) return st;
    st = gbt::with_elem(elem, [](auto v) { return gbt::prepare<decltype(v)>(); });
    if (st != GEMM_OK) return st;
    void* word = nullptr;
    const size_t sums = gbt::fits(vocab, gbt::elem_bytes(elem)) ? 0 : static_cast<size_t>(max_rows) * sizeof(float2);
    st = gbt::allocate(&word, 256 + sums);
    if (st != GEMM_OK) return st;
    gemm_distill_plan* p = new (std::nothrow) gemm_distill_plan();
    if (!p || gbt::clear_now(word, 256) != GEMM_OK) {
        cudaFree(word);
        st = p ? GEMM_ERR_CUDA : GEMM_ERR_OOM;
        delete p;
        return st;
    }
    p->max_rows = max_rows;
    p->vocab = vocab;
    p->max_top = max_top;
    p->elem = elem;
    p->device = device;
    p->num_sms = sms;
    p->error_word = static_cast<int32_t*>(word);
    p->sums = reinterpret_cast<float2*>(static_cast<uint8_t*>(word) + 256);
    gbt::with_elem(elem, [&](auto v) {
        p->forward = gbt::stream_shape<decltype(v), gbt::kForward>(vocab, max_top);
        p->both = gbt::stream_shape<decltype(v), gbt::kBoth>(vocab, max_top);
        return GEMM_OK;
    });
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_distill_forward(gemm_distill_plan_t p, int64_t rows, const void* logits,
                                   int64_t ldl, const gemm_teacher_t* teacher, float temperature,
                                   float* loss, float* lse, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    const gbt::Queue queue{stream, p->device};
    if (rows > 0 && (!loss || !lse)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(loss, 4) || !gbt::aligned(lse, 4)) return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    return gbt::with_elem(p->elem, [&](auto v) {
        using T = decltype(v);
        auto a = gbt::arguments<T>(p, logits, ldl, teacher, temperature);
        a.loss = loss;
        a.lse = lse;
        if (p->forward.clusters > 0 && rows >= p->forward.clusters)
            return gbt::run_stream<T, gbt::kForward>(a, p->forward, rows, queue);
        return gbt::fits(p->vocab, sizeof(T)) ? gbt::run<T, gbt::kForward>(a, rows, p->num_sms, queue)
                                              : gbt::run_forward_wide(a, rows, queue);
    });
}

gemm_status_t gemm_distill_backward(gemm_distill_plan_t p, int64_t rows, const void* logits,
                                    int64_t ldl, const gemm_teacher_t* teacher, float temperature,
                                    const float* lse, const float* dloss, void* dlogits,
                                    int64_t ldd, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    const gbt::Queue queue{stream, p->device};
    if (rows > 0 && (!lse || !dlogits || ldd < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(lse, 4) || !gbt::aligned(dloss, 4) ||
        !gbt::aligned(dlogits, gbt::elem_bytes(p->elem)))
        return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    return gbt::with_elem(p->elem, [&](auto v) {
        using T = decltype(v);
        auto a = gbt::arguments<T>(p, logits, ldl, teacher, temperature);
        a.lse = const_cast<float*>(lse);     // (read only)
        a.dloss = dloss;
        a.dlogits = static_cast<T*>(dlogits);
        a.ldd = ldd;
        return gbt::run<T, gbt::kBackward>(a, rows, p->num_sms, queue);
    });
}

gemm_status_t gemm_distill_forward_backward(gemm_distill_plan_t p, int64_t rows,
                                            const void* logits, int64_t ldl,
                                            const gemm_teacher_t* teacher, float temperature,
                                            const float* dloss, float* loss, float* lse,
                                            void* dlogits, int64_t ldd, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    const gbt::Queue queue{stream, p->device};
    if (rows > 0 && (!loss || !lse || !dlogits || ldd < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(loss, 4) || !gbt::aligned(lse, 4) || !gbt::aligned(dloss, 4) ||
        !gbt::aligned(dlogits, gbt::elem_bytes(p->elem)))
        return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    return gbt::with_elem(p->elem, [&](auto v) {
        using T = decltype(v);
        auto a = gbt::arguments<T>(p, logits, ldl, teacher, temperature);
        a.loss = loss;
        a.lse = lse;
        a.dloss = dloss;
        a.dlogits = static_cast<T*>(dlogits);
        a.ldd = ldd;
        if (p->both.clusters > 0 && rows >= p->both.clusters)
            return gbt::run_stream<T, gbt::kBoth>(a, p->both, rows, queue);
        if (gbt::fits(p->vocab, sizeof(T))) return gbt::run<T, gbt::kBoth>(a, rows, p->num_sms, queue);
        a.sums = p->sums;
        const gemm_status_t first = gbt::run_forward_wide(a, rows, queue);
        return first == GEMM_OK ? gbt::run<T, gbt::kBackward>(a, rows, p->num_sms, queue) : first;
    });
}

gemm_status_t gemm_distill_plan_set_timeout(gemm_distill_plan_t p, uint64_t ns) {
    return p ? gbt::set_wait_limit(&p->waits, ns) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_distill_plan_set_wait_test(gemm_distill_plan_t p, uint32_t extra_bytes, uint32_t every) {
    return p ? gbt::set_wait_test(&p->waits, extra_bytes, every) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_distill_plan_check(gemm_distill_plan_t p, void* stream) {
    return p ? gbt::check_error_word(p->error_word, stream) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_distill_plan_destroy(gemm_distill_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->error_word) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
