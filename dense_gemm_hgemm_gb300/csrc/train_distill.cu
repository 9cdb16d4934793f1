// train_distill.cu -- the distillation loss of gemm_train.h against a teacher's top
// logits, forward and backward.
#include <math.h>

#include <new>

#include "train_common.cuh"

struct gemm_distill_plan {
    int64_t max_rows, vocab, max_top;
    gemm_elem_t elem;
    int device, num_sms;
    int32_t* error_word;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct Teacher {
    const void* ids;
    const void* values;
    const float* lse;
    int64_t ld_ids, ld_values;
    int top, id_type, value_elem;
};

// A row's teacher entries in shared memory: ids (-1 = no entry), log2 of the
// probabilities and the probabilities; `mass` is their sum.
struct Entries {
    int32_t id[kMaxTop];
    float log2p[kMaxTop];
    float p[kMaxTop];
    float part[kThreads / 32];
    float mass;
};

__device__ float block_reduce(float v, bool is_max, float* part) {
    v = is_max ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
    for (int w = 1; w < kThreads / 32; ++w) v = is_max ? fmaxf(v, part[w]) : v + part[w];
    return v;
}

// Scaled logits are kept as log2 values: c = log2(e) / temperature.
__device__ void load_entries(Entries& en, const Teacher& t, int64_t row, float c, int64_t vocab,
                             int32_t* error) {
    float high = -INFINITY, sum = 0.f;
    for (int j = threadIdx.x; j < t.top; j += kThreads) {
        int64_t id = load_index(t.ids, row * t.ld_ids + j, t.id_type);
        if (id >= vocab) {
            *error = 1;
            id = -1;
        }
        const float v = id < 0 ? -INFINITY : load_elem(t.values, row * t.ld_values + j, t.value_elem) * c;
        en.id[j] = id < 0 ? -1 : static_cast<int32_t>(id);
        en.log2p[j] = v;
        high = fmaxf(high, v);
    }
    high = block_reduce(high, true, en.part);
    float norm;
    if (t.lse) {
        norm = t.lse[row] * kLog2e;
    } else {
        for (int j = threadIdx.x; j < t.top; j += kThreads)
            sum += en.log2p[j] == -INFINITY ? 0.f : exp2f(en.log2p[j] - high);
        norm = high + log2f(block_reduce(sum, false, en.part));
    }
    sum = 0.f;
    for (int j = threadIdx.x; j < t.top; j += kThreads) {
        const float l = en.log2p[j] == -INFINITY ? -INFINITY : en.log2p[j] - norm;
        en.log2p[j] = l;
        en.p[j] = exp2f(l);
        sum += en.p[j];
    }
    sum = block_reduce(sum, false, en.part);
    if (threadIdx.x == 0) en.mass = sum;
    __syncthreads();
}

// One block a row: the row's maximum, the sum, the loss over the teacher's entries.
template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_forward_kernel(const T* logits, int64_t ldl, Teacher t, float temperature, int vocab,
                       float* loss, float* lse, int32_t* error) {
    __shared__ Entries en;
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* s = logits + row * ldl;
    const float c = kLog2e / temperature;
    load_entries(en, t, row, c, vocab, error);
    if (en.mass == 0.f) {
        if (threadIdx.x == 0) {
            loss[row] = 0.f;
            lse[row] = -INFINITY;
        }
        return;
    }
    float high = -INFINITY, sum = 0.f;
    for (int i = threadIdx.x; i < vocab; i += kThreads) high = fmaxf(high, to_f32(s[i]));
    high = block_reduce(high, true, en.part);
    const float base = high == -INFINITY ? 0.f : high * c;
    for (int i = threadIdx.x; i < vocab; i += kThreads) sum += exp2f(to_f32(s[i]) * c - base);
    sum = block_reduce(sum, false, en.part);
    const float l2 = base + log2f(sum);
    float total = 0.f;
    for (int j = threadIdx.x; j < t.top; j += kThreads)
        if (!(en.p[j] == 0.f)) total += en.p[j] * (en.log2p[j] - to_f32(s[en.id[j]]) * c + l2);
    total = block_reduce(total, false, en.part);
    if (threadIdx.x == 0) {
        const bool empty = sum == 0.f;
        loss[row] = empty ? 0.f : temperature * temperature * total / kLog2e;
        lse[row] = empty ? -INFINITY : l2 / kLog2e;
    }
}

// One block a row: P * q over the row, then the teacher's entries.
template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_backward_kernel(const T* logits, int64_t ldl, Teacher t, float temperature, int vocab,
                        const float* lse, const float* dloss, T* dlogits, int64_t ldd,
                        int32_t* error) {
    __shared__ Entries en;
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* s = logits + row * ldl;
    T* d = dlogits + row * ldd;
    const float c = kLog2e / temperature;
    load_entries(en, t, row, c, vocab, error);
    const float l2 = lse[row] * kLog2e;
    if (en.mass == 0.f || l2 == -INFINITY) {
        for (int i = threadIdx.x; i < vocab; i += kThreads) d[i] = from_f32<T>(0.f);
        return;
    }
    const float scale = temperature * (dloss ? dloss[row] : 1.f);
    // the entries' own gradients, before dlogits overwrites the logits: the first
    // entry of each id takes them all
    __shared__ float own[kMaxTop];
    for (int j = threadIdx.x; j < t.top; j += kThreads) {
        if (en.id[j] < 0) continue;
        float p = 0.f;
        for (int k = 0; k < t.top; ++k)
            if (en.id[k] == en.id[j]) p += en.p[k];
        own[j] = scale * (en.mass * exp2f(to_f32(s[en.id[j]]) * c - l2) - p);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < vocab; i += kThreads)
        d[i] = from_f32<T>(scale * en.mass * exp2f(to_f32(s[i]) * c - l2));
    __syncthreads();
    for (int j = threadIdx.x; j < t.top; j += kThreads)
        if (en.id[j] >= 0) d[en.id[j]] = from_f32<T>(own[j]);   // equal ids write equal values
}

gemm_status_t check_call(const gemm_distill_plan* p, int64_t rows, const void* logits, int64_t ldl,
                         const gemm_teacher_t* t, float temperature) {
    if (!p || rows < 0 || rows > p->max_rows || !t) return GEMM_ERR_INVALID_ARG;
    if (!valid_index(t->id_type) || !valid_elem(t->value_elem)) return GEMM_ERR_UNSUPPORTED;
    if (!(temperature > 0.f) || t->top < 0 || t->top > p->max_top) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && (!logits || ldl < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && t->top > 0 &&
        (!t->ids || !t->values || t->ld_ids < t->top || t->ld_values < t->top))
        return GEMM_ERR_INVALID_ARG;
    if (!aligned(logits, elem_bytes(p->elem)) || !aligned(t->ids, index_bytes(t->id_type)) ||
        !aligned(t->values, elem_bytes(t->value_elem)) || !aligned(t->lse, 4))
        return GEMM_ERR_ALIGNMENT;
    return check_device(p->device);
}

Teacher device_teacher(const gemm_teacher_t* t) {
    return Teacher{t->ids,       t->values,
                   t->lse,       t->ld_ids,
                   t->ld_values, static_cast<int>(t->top),
                   static_cast<int>(t->id_type), static_cast<int>(t->value_elem)};
}

}  // namespace
}  // namespace gbt

extern "C" {

gemm_status_t gemm_distill_plan_create(int64_t max_rows, int64_t vocab, int64_t max_top,
                                       gemm_elem_t elem, gemm_distill_plan_t* plan) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!gbt::valid_elem(elem)) return GEMM_ERR_UNSUPPORTED;
    if (max_rows < 0 || max_rows > INT32_MAX || vocab < 1 || vocab > INT32_MAX || max_top < 0 ||
        max_top > gbt::kMaxTop)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    gemm_status_t st = gbt::current_device(&device, &sms);
    if (st != GEMM_OK) return st;
    void* word = nullptr;
    st = gbt::allocate(&word, 256);
    if (st != GEMM_OK) return st;
    gemm_distill_plan* p = new (std::nothrow) gemm_distill_plan();
    if (!p || cudaMemset(word, 0, 256) != cudaSuccess) {
        cudaGetLastError();
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
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_distill_forward(gemm_distill_plan_t p, int64_t rows, const void* logits,
                                   int64_t ldl, const gemm_teacher_t* teacher, float temperature,
                                   float* loss, float* lse, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    if (rows > 0 && (!loss || !lse)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(loss, 4) || !gbt::aligned(lse, 4)) return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    return gbt::with_elem(p->elem, [&](auto v) {
        using T = decltype(v);
        return gbt::launch(gbt::distill_forward_kernel<T>, rows, gbt::kThreads, 0, stream, 1,
                           static_cast<const T*>(logits), ldl, gbt::device_teacher(teacher),
                           temperature, static_cast<int>(p->vocab), loss, lse, p->error_word);
    });
}

gemm_status_t gemm_distill_backward(gemm_distill_plan_t p, int64_t rows, const void* logits,
                                    int64_t ldl, const gemm_teacher_t* teacher, float temperature,
                                    const float* lse, const float* dloss, void* dlogits,
                                    int64_t ldd, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    if (rows > 0 && (!lse || !dlogits || ldd < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(lse, 4) || !gbt::aligned(dloss, 4) ||
        !gbt::aligned(dlogits, gbt::elem_bytes(p->elem)))
        return GEMM_ERR_ALIGNMENT;
    if (rows == 0) return GEMM_OK;
    return gbt::with_elem(p->elem, [&](auto v) {
        using T = decltype(v);
        return gbt::launch(gbt::distill_backward_kernel<T>, rows, gbt::kThreads, 0, stream, 1,
                           static_cast<const T*>(logits), ldl, gbt::device_teacher(teacher),
                           temperature, static_cast<int>(p->vocab), lse, dloss,
                           static_cast<T*>(dlogits), ldd, p->error_word);
    });
}

gemm_status_t gemm_distill_forward_backward(gemm_distill_plan_t p, int64_t rows,
                                            const void* logits, int64_t ldl,
                                            const gemm_teacher_t* teacher, float temperature,
                                            const float* dloss, float* loss, float* lse,
                                            void* dlogits, int64_t ldd, void* stream) {
    const gemm_status_t st = gbt::check_call(p, rows, logits, ldl, teacher, temperature);
    if (st != GEMM_OK) return st;
    if (rows > 0 && (!loss || !lse || !dlogits || ldd < p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(loss, 4) || !gbt::aligned(lse, 4) || !gbt::aligned(dloss, 4) ||
        !gbt::aligned(dlogits, gbt::elem_bytes(p->elem)))
        return GEMM_ERR_ALIGNMENT;
    const gemm_status_t first =
        gemm_distill_forward(p, rows, logits, ldl, teacher, temperature, loss, lse, stream);
    if (first != GEMM_OK) return first;
    return gemm_distill_backward(p, rows, logits, ldl, teacher, temperature, lse, dloss, dlogits,
                                 ldd, stream);
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
