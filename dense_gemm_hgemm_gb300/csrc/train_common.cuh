// train_common.cuh -- what the kernels of gemm_train.h share: element types,
// reductions, the launch (programmatic dependent launch on the caller's stream)
// and the host-side checks.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "gemm_train.h"

namespace gbt {

// The longest rows a plan takes: column counters are 32-bit and run a step past the end.
constexpr int64_t kMostColumns = int64_t{1} << 30;

// ---- element types ------------------------------------------------------------

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// An element of a matrix whose type is known at run time (small operands only).
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int elem) {
    if (elem == GEMM_ELEM_F32) return static_cast<const float*>(p)[i];
    if (elem == GEMM_ELEM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int type) {
    return type == GEMM_INDEX_I64 ? static_cast<const int64_t*>(p)[i]
                                  : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}

// ---- packs: VEC elements that move as one access --------------------------------

template <int BYTES> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <typename T, int VEC>
struct Pack {
    typename RawOf<static_cast<int>(sizeof(T)) * VEC>::type raw;
    __device__ __forceinline__ float get(int i) const {
        return to_f32(reinterpret_cast<const T*>(&raw)[i]);
    }
    __device__ __forceinline__ void set(int i, float v) {
        reinterpret_cast<T*>(&raw)[i] = from_f32<T>(v);
    }
    __device__ __forceinline__ void set_raw(int i, T v) { reinterpret_cast<T*>(&raw)[i] = v; }
    __device__ __forceinline__ void clear() { raw = {}; }
};

// ---- pairs of fp32 values, which one instruction works on -------------------------

struct Pair {
    uint64_t bits;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float lo, float hi) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(lo), "f"(hi));
    }
    __device__ __forceinline__ void get(float& lo, float& hi) const {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(bits));
    }
};

__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits), "l"(c.bits));
    return d;
}

__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits));
    return d;
}

__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.bits) : "l"(a.bits), "l"(b.bits));
    return d;
}

// Elements 2j and 2j + 1 of a pack, and back (rounded once).
template <int VEC>
__device__ __forceinline__ Pair pair_of(const Pack<float, VEC>& q, int j) {
    const float* f = reinterpret_cast<const float*>(&q.raw);
    return Pair(f[2 * j], f[2 * j + 1]);
}
template <int VEC>
__device__ __forceinline__ Pair pair_of(const Pack<__half, VEC>& q, int j) {
    const float2 f = __half22float2(reinterpret_cast<const __half2*>(&q.raw)[j]);
    return Pair(f.x, f.y);
}
template <int VEC>
__device__ __forceinline__ Pair pair_of(const Pack<__nv_bfloat16, VEC>& q, int j) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&q.raw)[j];
    return Pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <int VEC>
__device__ __forceinline__ void set_pair(Pack<float, VEC>& q, int j, Pair v) {
    float* f = reinterpret_cast<float*>(&q.raw);
    v.get(f[2 * j], f[2 * j + 1]);
}
template <int VEC>
__device__ __forceinline__ void set_pair(Pack<__half, VEC>& q, int j, Pair v) {
    float lo, hi;
    v.get(lo, hi);
    reinterpret_cast<__half2*>(&q.raw)[j] = __floats2half2_rn(lo, hi);
}
template <int VEC>
__device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, VEC>& q, int j, Pair v) {
    float lo, hi;
    v.get(lo, hi);
    reinterpret_cast<__nv_bfloat162*>(&q.raw)[j] = __floats2bfloat162_rn(lo, hi);
}

// All elements of some packs as pairs, and back (an even number of packs of one element
// each, else pairs within the packs).
template <typename T, int VEC, int PACKS>
__device__ __forceinline__ void to_pairs(const Pack<T, VEC> (&p)[PACKS], Pair (&v)[PACKS * VEC / 2]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int j = 0; j < PACKS / 2; ++j) v[j] = Pair(p[2 * j].get(0), p[2 * j + 1].get(0));
    } else {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) v[k * (VEC / 2) + j] = pair_of(p[k], j);
        }
    }
}

template <typename T, int VEC, int PACKS>
__device__ __forceinline__ void from_pairs(const Pair (&v)[PACKS * VEC / 2], Pack<T, VEC> (&p)[PACKS]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int j = 0; j < PACKS / 2; ++j) {
            float lo, hi;
            v[j].get(lo, hi);
            p[2 * j].set(0, lo);
            p[2 * j + 1].set(0, hi);
        }
    } else {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) set_pair(p[k], j, v[k * (VEC / 2) + j]);
        }
    }
}

// The largest of some packs' elements (NaN aside).
template <int VEC, int N>
__device__ __forceinline__ float pack_max(const Pack<float, VEC> (&q)[N]) {
    float m = reinterpret_cast<const float*>(&q[0].raw)[0];
#pragma unroll
    for (int b = 0; b < N; ++b) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, reinterpret_cast<const float*>(&q[b].raw)[i]);
    }
    return m;
}
template <typename T2, int WORDS, typename P, int N>
__device__ __forceinline__ T2 word_max(const P (&q)[N]) {
    T2 m = reinterpret_cast<const T2*>(&q[0].raw)[0];
#pragma unroll
    for (int b = 0; b < N; ++b) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) m = __hmax2(m, reinterpret_cast<const T2*>(&q[b].raw)[i]);
    }
    return m;
}
template <int VEC, int N>
__device__ __forceinline__ float pack_max(const Pack<__half, VEC> (&q)[N]) {
    const float2 f = __half22float2(word_max<__half2, VEC / 2>(q));
    return fmaxf(f.x, f.y);
}
template <int VEC, int N>
__device__ __forceinline__ float pack_max(const Pack<__nv_bfloat16, VEC> (&q)[N]) {
    const float2 f = __bfloat1622float2(word_max<__nv_bfloat162, VEC / 2>(q));
    return fmaxf(f.x, f.y);
}

// The first n of VEC elements at p (the rest zeros); p is aligned to the pack.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p, int64_t n) {
    using Raw = decltype(Pack<T, VEC>::raw);
    Pack<T, VEC> r;
    if (n >= VEC) {
        r.raw = *reinterpret_cast<const Raw*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.set_raw(i, i < n ? p[i] : from_f32<T>(0.f));
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, int64_t n, const Pack<T, VEC>& v) {
    using Raw = decltype(Pack<T, VEC>::raw);
    if (n >= VEC) {
        *reinterpret_cast<Raw*>(p) = v.raw;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n) p[i] = reinterpret_cast<const T*>(&v.raw)[i];
    }
}

// VEC fp32 values as elements of G (several accesses where they are wider than 16 bytes).
template <typename G, int VEC>
__device__ __forceinline__ void load_values(const G* p, int64_t n, float (&v)[VEC]) {
    constexpr int kPer = VEC * static_cast<int>(sizeof(G)) > 16 ? 16 / static_cast<int>(sizeof(G)) : VEC;
#pragma unroll
    for (int k = 0; k < VEC; k += kPer) {
        const Pack<G, kPer> q = load_pack<G, kPer>(p + k, n - k);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[k + i] = q.get(i);
    }
}

template <typename G, int VEC>
__device__ __forceinline__ void store_values(G* p, int64_t n, const float (&v)[VEC]) {
    constexpr int kPer = VEC * static_cast<int>(sizeof(G)) > 16 ? 16 / static_cast<int>(sizeof(G)) : VEC;
#pragma unroll
    for (int k = 0; k < VEC; k += kPer) {
        Pack<G, kPer> q;
#pragma unroll
        for (int i = 0; i < kPer; ++i) q.set(i, v[k + i]);
        store_pack<G, kPer>(p + k, n - k, q);
    }
}

// 2^v to two units in the last place (results below 2^-126 are zero).
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---- reductions ---------------------------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The previous kernel of the stream has finished and its writes are visible.
__device__ __forceinline__ void wait_for_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The next kernel of the stream may be brought up (it waits as above itself).
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// All threads of the cluster; writes before it, to global memory too, are visible after it.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- asynchronous copies into a ring of buffers ------------------------------------

constexpr uint32_t kWaitNs = 2000000000u;       // the longest wait in a kernel, by default
constexpr uint32_t kNoticeNs = 20000;           // ... and the shortest: no limit is looked at before

// A plan's limit of a wait, and its test hook: bytes that the copies of every `every`-th block
// wait for beyond what they bring.
struct Waits {
    uint32_t limit = kWaitNs;            // ns, by the timer's lower word (which wraps after 4.29 s)
    uint32_t extra = 0, every = 1;
    __device__ __forceinline__ uint32_t extra_bytes() const {
        return extra == 0 || blockIdx.x % every != every - 1 ? 0 : extra;
    }
};

constexpr int32_t kErrorIndex = 1;              // bits of a plan's error word
constexpr int32_t kErrorTimeout = 2;

__device__ __forceinline__ uint32_t shared_address(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint32_t timer_ns() {
    uint32_t now;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
    return now;
}

// Waits for a phase of the barrier, at most `limit` ns.
__device__ inline bool wait_phase(uint64_t* barrier, uint32_t parity, uint32_t limit) {
    const uint32_t at = shared_address(barrier);
    uint32_t began = 0;
    for (uint32_t tries = 0;; ++tries) {
        uint32_t done;
        asm volatile(
            "{\n.reg .pred p;\n"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done) : "r"(at), "r"(parity) : "memory");
        if (done) return true;
        const uint32_t now = timer_ns();
        if (tries == 0) began = now;
        if (now - began > kNoticeNs && now - began > limit) return false;
    }
}

// Waits for a phase of the barrier until `limit` ns after `began`: several waits within one limit.
__device__ inline void wait_until(uint64_t* barrier, uint32_t parity, uint32_t began, uint32_t limit) {
    const uint32_t spent = timer_ns() - began;
    if (spent < limit) wait_phase(barrier, parity, limit - spent);
}

// A place in a ring of buffers, and how often it has been passed.
struct Turn {
    int at;
    uint32_t round;
    __device__ __forceinline__ void next(int by, int size) {
        for (at += by; at >= size; at -= size) ++round;
    }
};

// As wait_phase, for whole warps, at most *patience ns.  When it runs out, *patience becomes 0;
// later waits with it last kNoticeNs at most.  (The patience is looked at after that time only:
// a limit in a register, or one read from shared memory at each try, cost 1% of the time of
// distillation's pipeline.)
__device__ __forceinline__ bool wait_or_die(uint64_t* barrier, uint32_t parity, uint32_t* patience, int32_t* error) {
    const uint32_t at = shared_address(barrier);
    uint32_t began = 0;
    for (uint32_t tries = 0;; ++tries) {
        uint32_t done;
        asm volatile(
            "{\n.reg .pred p;\n"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done) : "r"(at), "r"(parity) : "memory");
        if (done) return true;
        const uint32_t now = timer_ns();
        if (tries == 0) began = now;
        if (now - began <= kNoticeNs) continue;
        const uint32_t limit = *static_cast<volatile uint32_t*>(patience);
        if (limit == 0) return false;
        if (now - began > limit) {
            *static_cast<volatile uint32_t*>(patience) = 0;
            atomicOr(error, kErrorTimeout);
            return false;
        }
    }
}

// Whether waits with this patience have been given up.
__device__ __forceinline__ bool is_dead(const uint32_t* patience) {
    return *static_cast<const volatile uint32_t*>(patience) == 0;
}

__device__ __forceinline__ void init_barrier(uint64_t* barrier, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(shared_address(barrier)), "r"(count) : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* barrier) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(shared_address(barrier)) : "memory");
}

// The barrier's phase ends when these bytes have come (and this was the last arrival);
// bytes (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void expect_bytes(uint64_t* barrier, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                 :: "r"(shared_address(barrier)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_bytes(void* to, const void* from, uint32_t bytes, uint64_t* barrier) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(shared_address(to)), "l"(from), "r"(bytes), "r"(shared_address(barrier)) : "memory");
}

// ---- host ---------------------------------------------------------------------

inline gemm_status_t set_wait_limit(Waits* w, uint64_t ns) {
    constexpr uint64_t kMost = 4000000000u;
    w->limit = ns == 0 ? kWaitNs : static_cast<uint32_t>(ns < kNoticeNs ? kNoticeNs : ns < kMost ? ns : kMost);
    return GEMM_OK;
}

inline gemm_status_t set_wait_test(Waits* w, uint32_t extra_bytes, uint32_t every) {
    if (extra_bytes > 4096 || extra_bytes % 16 != 0 || every == 0) return GEMM_ERR_INVALID_ARG;
    w->extra = extra_bytes;
    w->every = every;
    return GEMM_OK;
}

inline bool valid_elem(gemm_elem_t e) { return e >= GEMM_ELEM_F16 && e <= GEMM_ELEM_F32; }
inline int elem_bytes(gemm_elem_t e) { return e == GEMM_ELEM_F32 ? 4 : 2; }
inline bool valid_index(gemm_index_t t) { return t == GEMM_INDEX_I32 || t == GEMM_INDEX_I64; }
inline int index_bytes(gemm_index_t t) { return t == GEMM_INDEX_I64 ? 8 : 4; }
inline bool aligned(const void* p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

// How many plans have been made.
inline std::atomic<uint32_t>& plans_made() {
    static std::atomic<uint32_t> n{0};
    return n;
}

// A plan is about to be made: the current device and its SMs.
inline gemm_status_t begin_plan(int* device, int* num_sms) {
    int dev = -1, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (major != 10 || minor != 3) return GEMM_ERR_ARCH;
    plans_made().fetch_add(1, std::memory_order_release);
    *device = dev;
    return GEMM_OK;
}

inline gemm_status_t check_device(int device) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    return dev == device ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

inline gemm_status_t allocate(void** p, size_t bytes) {
    if (cudaMalloc(p, bytes) == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    *p = nullptr;
    return GEMM_ERR_OOM;
}

// Zeros, written before it returns whatever the default stream has queued (a memset there could
// clear an error word after a kernel on another stream has set it).
inline gemm_status_t clear_now(void* p, size_t bytes) {
    cudaStream_t stream;
    if (cudaStreamCreateWithFlags(&stream, cudaStreamNonBlocking) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    const bool ok = cudaMemsetAsync(p, 0, bytes, stream) == cudaSuccess && cudaStreamSynchronize(stream) == cudaSuccess;
    if (cudaStreamDestroy(stream) == cudaSuccess && ok) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_CUDA;
}

// Synchronise, then read and clear an error word, all on the stream.
inline gemm_status_t check_error_word(int32_t* word, void* stream_ptr) {
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    int32_t value = 0;
    if (cudaMemcpyAsync(&value, word, sizeof(value), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess ||
        (value != 0 && (cudaMemsetAsync(word, 0, sizeof(value), stream) != cudaSuccess ||
                        cudaStreamSynchronize(stream) != cudaSuccess))) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    if (value & kErrorTimeout) return GEMM_ERR_DEVICE_TIMEOUT;
    return value != 0 ? GEMM_ERR_INDEX : GEMM_OK;
}

// Rows of a matrix start at multiples of 16 bytes (so whole packs can move).
inline bool rows_aligned(const void* p, int64_t ld, int bytes) {
    return aligned(p, 16) && (ld * bytes) % 16 == 0;
}

// Where a call's kernels go: the caller's stream, on the plan's device.
struct Queue {
    void* stream;
    int device;
};

// cuLaunchKernelEx, which with a kernel's function handle costs 0.4 us less host time a call
// than the runtime's launch of its stub.
inline PFN_cuLaunchKernelEx_v11060 driver_launch() {
    static PFN_cuLaunchKernelEx_v11060 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuLaunchKernelEx", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuLaunchKernelEx_v11060>(p);
    });
    return fn;
}

// The kernel's function handle on the device (which is current), looked up once after each
// plan's creation: handles do not outlive a context, and neither do plans.
template <auto Kernel>
CUfunction function_of(int device) {
    constexpr int kDevices = 16;
    static std::atomic<CUfunction> known[kDevices];
    static std::atomic<uint32_t> known_at[kDevices];
    const bool kept = device >= 0 && device < kDevices;
    const uint32_t now = plans_made().load(std::memory_order_acquire);
    CUfunction fn = nullptr;
    if (kept && known_at[device].load(std::memory_order_acquire) == now)
        fn = known[device].load(std::memory_order_relaxed);
    if (!fn) {
        cudaFunction_t f = nullptr;
        if (cudaGetFuncBySymbol(&f, reinterpret_cast<const void*>(Kernel)) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        fn = reinterpret_cast<CUfunction>(f);
        if (kept) {
            known[device].store(fn, std::memory_order_relaxed);
            known_at[device].store(now, std::memory_order_release);
        }
    }
    return fn;
}

template <typename T> struct Same { using type = T; };

template <typename... P>
CUresult fire(void (*)(P...), const CUlaunchConfig& cfg, CUfunction fn, typename Same<P>::type... args) {
    void* pointers[] = {static_cast<void*>(&args)...};
    return driver_launch()(&cfg, fn, pointers, nullptr);
}

// Launch with programmatic dependent launch: the kernel starts its first
// instructions while the stream's previous kernel ends, and calls
// wait_for_previous_kernel before it touches memory.
template <auto Kernel, typename... A>
gemm_status_t launch(int64_t grid, int block, size_t smem, Queue queue, int cluster, A... args) {
    const CUfunction fn = function_of<Kernel>(queue.device);
    if (!fn || !driver_launch() || grid > INT32_MAX) return GEMM_ERR_LAUNCH;
    CUlaunchAttribute attr[2];
    attr[0].id = CU_LAUNCH_ATTRIBUTE_PROGRAMMATIC_STREAM_SERIALIZATION;
    attr[0].value.programmaticStreamSerializationAllowed = 1;
    attr[1].id = CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION;
    attr[1].value.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].value.clusterDim.y = 1;
    attr[1].value.clusterDim.z = 1;
    CUlaunchConfig cfg = {};
    cfg.gridDimX = static_cast<unsigned>(grid);
    cfg.gridDimY = cfg.gridDimZ = 1;
    cfg.blockDimX = static_cast<unsigned>(block);
    cfg.blockDimY = cfg.blockDimZ = 1;
    cfg.sharedMemBytes = static_cast<unsigned>(smem);
    cfg.hStream = static_cast<CUstream>(queue.stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    CUresult r = fire(Kernel, cfg, fn, args...);
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaSetDevice(queue.device) == cudaSuccess)
        r = fire(Kernel, cfg, fn, args...);              // a thread without a current context
    return r == CUDA_SUCCESS ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// Calls f with a value of the element type.
template <typename F>
gemm_status_t with_elem(gemm_elem_t e, F f) {
    if (e == GEMM_ELEM_F16) return f(__half());
    if (e == GEMM_ELEM_BF16) return f(__nv_bfloat16());
    return f(float());
}

}  // namespace gbt
