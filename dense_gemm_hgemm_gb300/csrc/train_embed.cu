// train_embed.cu -- embedding lookup of gemm_train.h and its table's gradient.
#include <new>

#include "train_common.cuh"

struct gemm_embed_plan {
    int64_t vocab, dim, max_tokens;
    gemm_elem_t elem, grad_elem;
    int device, num_sms;
    int32_t* error_word;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;

// One block a token.
template <typename T>
__global__ void __launch_bounds__(kThreads)
embed_forward_kernel(const void* ids, int id_type, int64_t padding, const T* table, int64_t ldt,
                     float scale, T* out, int64_t ldo, int64_t vocab, int dim, int32_t* error) {
    wait_for_previous_kernel();
    const int64_t t = blockIdx.x;
    const int64_t id = load_index(ids, t, id_type);
    const bool inside = id >= 0 && id < vocab;
    if (!inside && id != padding && threadIdx.x == 0) *error = 1;
    const bool take = inside && id != padding;
    for (int c = threadIdx.x; c < dim; c += kThreads)
        out[t * ldo + c] = from_f32<T>(take ? scale * to_f32(table[id * ldt + c]) : 0.f);
}

// One block a table row: it goes through all ids, in order.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads)
embed_backward_kernel(const void* ids, int id_type, int64_t padding, const T* dout, int64_t ldo,
                      float scale, G* dtable, int64_t ldt, int accumulate, int64_t tokens,
                      int64_t vocab, int dim, int32_t* error) {
    wait_for_previous_kernel();
    const int64_t v = blockIdx.x;
    __shared__ int32_t found[kThreads];
    __shared__ int count;
    for (int64_t c0 = 0; c0 < dim; c0 += kThreads) {
        const int64_t c = c0 + threadIdx.x;
        float sum = 0.f;
        int any = 0;
        for (int64_t t0 = 0; t0 < tokens; t0 += kThreads) {
            const int64_t t = t0 + threadIdx.x;
            const int64_t id = t < tokens ? load_index(ids, t, id_type) : padding;
            const bool mine = id == v && id != padding;
            if (v == 0 && t < tokens && id != padding && (id < 0 || id >= vocab)) *error = 1;
            if (!__syncthreads_or(mine)) continue;
            if (threadIdx.x == 0) count = 0;
            for (int w = 0; w < kThreads / 32; ++w) {   // the matches in order
                __syncthreads();
                if (threadIdx.x / 32 == w) {
                    const unsigned m = __ballot_sync(0xffffffffu, mine);
                    const int lane = threadIdx.x % 32;
                    if (mine) found[count + __popc(m & ((1u << lane) - 1u))] = static_cast<int32_t>(t);
                    __syncwarp();
                    if (lane == 0) count += __popc(m);
                }
            }
            __syncthreads();
            any = 1;
            if (c < dim)
                for (int k = 0; k < count; ++k) sum += to_f32(dout[found[k] * ldo + c]);
            __syncthreads();
        }
        if (c < dim) {
            G* at = dtable + v * ldt + c;
            if (!accumulate) *at = from_f32<G>(scale * sum);
            else if (any) *at = from_f32<G>(to_f32(*at) + scale * sum);
        }
    }
}

}  // namespace
}  // namespace gbt

extern "C" {

gemm_status_t gemm_embed_plan_create(int64_t vocab, int64_t dim, int64_t max_tokens,
                                     gemm_elem_t elem, gemm_elem_t grad_elem,
                                     gemm_embed_plan_t* plan) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if (!gbt::valid_elem(elem) || (grad_elem != elem && grad_elem != GEMM_ELEM_F32))
        return GEMM_ERR_UNSUPPORTED;
    if (vocab < 1 || vocab > INT32_MAX || dim < 1 || dim > INT32_MAX || max_tokens < 0 ||
        max_tokens > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    gemm_status_t st = gbt::current_device(&device, &sms);
    if (st != GEMM_OK) return st;
    void* word = nullptr;
    st = gbt::allocate(&word, 256);
    if (st != GEMM_OK) return st;
    gemm_embed_plan* p = new (std::nothrow) gemm_embed_plan();
    if (!p || cudaMemset(word, 0, 256) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(word);
        st = p ? GEMM_ERR_CUDA : GEMM_ERR_OOM;
        delete p;
        return st;
    }
    p->vocab = vocab;
    p->dim = dim;
    p->max_tokens = max_tokens;
    p->elem = elem;
    p->grad_elem = grad_elem;
    p->device = device;
    p->num_sms = sms;
    p->error_word = static_cast<int32_t*>(word);
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_embed_forward(gemm_embed_plan_t p, int64_t tokens, const void* ids,
                                 gemm_index_t id_type, int64_t padding, const void* table,
                                 int64_t ldt, float scale, void* out, int64_t ldo, void* stream) {
    if (!p || tokens < 0 || tokens > p->max_tokens) return GEMM_ERR_INVALID_ARG;
    if (!gbt::valid_index(id_type)) return GEMM_ERR_UNSUPPORTED;
    if (tokens > 0 && (!ids || !table || !out || ldt < p->dim || ldo < p->dim))
        return GEMM_ERR_INVALID_ARG;
    const int e = gbt::elem_bytes(p->elem);
    if (!gbt::aligned(ids, gbt::index_bytes(id_type)) || !gbt::aligned(table, e) ||
        !gbt::aligned(out, e))
        return GEMM_ERR_ALIGNMENT;
    const gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK || tokens == 0) return st;
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        return gbt::launch(gbt::embed_forward_kernel<T>, tokens, gbt::kThreads, 0, stream, 1, ids,
                           static_cast<int>(id_type), padding, static_cast<const T*>(table), ldt,
                           scale, static_cast<T*>(out), ldo, p->vocab, static_cast<int>(p->dim),
                           p->error_word);
    });
}

gemm_status_t gemm_embed_backward(gemm_embed_plan_t p, int64_t tokens, const void* ids,
                                  gemm_index_t id_type, int64_t padding, const void* dout,
                                  int64_t ldo, float scale, void* dtable, int64_t ldt,
                                  int32_t accumulate, void* stream) {
    if (!p || tokens < 0 || tokens > p->max_tokens || accumulate < 0 || accumulate > 1)
        return GEMM_ERR_INVALID_ARG;
    if (!gbt::valid_index(id_type)) return GEMM_ERR_UNSUPPORTED;
    if (!dtable || ldt < p->dim || (tokens > 0 && (!ids || !dout || ldo < p->dim)))
        return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(ids, gbt::index_bytes(id_type)) || !gbt::aligned(dout, gbt::elem_bytes(p->elem)) ||
        !gbt::aligned(dtable, gbt::elem_bytes(p->grad_elem)))
        return GEMM_ERR_ALIGNMENT;
    const gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK || (tokens == 0 && accumulate)) return st;
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        const auto run = [&](auto g) {
            using G = decltype(g);
            return gbt::launch(gbt::embed_backward_kernel<T, G>, p->vocab, gbt::kThreads, 0, stream,
                               1, ids, static_cast<int>(id_type), padding,
                               static_cast<const T*>(dout), ldo, scale, static_cast<G*>(dtable), ldt,
                               accumulate, tokens, p->vocab, static_cast<int>(p->dim),
                               p->error_word);
        };
        return p->grad_elem == GEMM_ELEM_F32 ? run(float()) : run(t);
    });
}

gemm_status_t gemm_embed_plan_check(gemm_embed_plan_t p, void* stream) {
    return p ? gbt::check_error_word(p->error_word, stream) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_embed_plan_destroy(gemm_embed_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->error_word) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
