// train_norm.cu -- layer norm of gemm_train.h, forward and backward.
#include <new>

#include "train_common.cuh"

struct gemm_norm_plan {
    int64_t max_rows, cols;
    gemm_elem_t elem, weight_elem;
    int device, num_sms;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;

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
__global__ void __launch_bounds__(kThreads)
norm_forward_kernel(const T* x, int64_t ldx, const W* gamma, const W* beta, float eps, T* y,
                    int64_t ldy, float* mean, float* rstd, int cols) {
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * ldx;
    T* yr = y + row * ldy;
    float s = 0.f;
    for (int c = threadIdx.x; c < cols; c += kThreads) s += to_f32(xr[c]);
    const float mu = block_sum(s) / static_cast<float>(cols);
    s = 0.f;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        const float d = to_f32(xr[c]) - mu;
        s += d * d;
    }
    const float r = 1.f / sqrtf(block_sum(s) / static_cast<float>(cols) + eps);
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        const float g = gamma ? to_f32(gamma[c]) : 1.f, b = beta ? to_f32(beta[c]) : 0.f;
        yr[c] = from_f32<T>((to_f32(xr[c]) - mu) * r * g + b);
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
}

// One block a row: the row's two sums, then dx.
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
norm_dx_kernel(const T* x, int64_t ldx, const W* gamma, const float* mean, const float* rstd,
               const T* dy, int64_t lddy, T* dx, int64_t lddx, int cols) {
    wait_for_previous_kernel();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * ldx;
    const T* dyr = dy + row * lddy;
    const float mu = mean[row], r = rstd[row];
    float sg = 0.f, sgx = 0.f;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        const float g = to_f32(dyr[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
        sg += g;
        sgx += g * ((to_f32(xr[c]) - mu) * r);
    }
    sg = block_sum(sg) / static_cast<float>(cols);
    sgx = block_sum(sgx) / static_cast<float>(cols);
    for (int c = threadIdx.x; c < cols; c += kThreads) {
        const float g = to_f32(dyr[c]) * (gamma ? to_f32(gamma[c]) : 1.f);
        dx[row * lddx + c] = from_f32<T>(r * (g - sg - (to_f32(xr[c]) - mu) * r * sgx));
    }
}

// One block per 32 columns: eight warps take every eighth row, then join.
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads)
norm_weight_grad_kernel(const T* x, int64_t ldx, const float* mean, const float* rstd, const T* dy,
                        int64_t lddy, int64_t rows, int cols, W* dgamma, W* dbeta) {
    __shared__ float part[2][kThreads / 32][32];
    wait_for_previous_kernel();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float dg = 0.f, db = 0.f;
    if (c < cols) {
        for (int64_t row = warp; row < rows; row += kThreads / 32) {
            const float d = to_f32(dy[row * lddy + c]);
            dg += d * ((to_f32(x[row * ldx + c]) - mean[row]) * rstd[row]);
            db += d;
        }
    }
    part[0][warp][lane] = dg;
    part[1][warp][lane] = db;
    __syncthreads();
    if (warp == 0 && c < cols) {
        dg = db = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) {
            dg += part[0][w][lane];
            db += part[1][w][lane];
        }
        if (dgamma) dgamma[c] = from_f32<W>(dg);
        if (dbeta) dbeta[c] = from_f32<W>(db);
    }
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
    if (max_rows < 0 || max_rows > INT32_MAX || cols < 1 || cols > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    const gemm_status_t st = gbt::current_device(&device, &sms);
    if (st != GEMM_OK) return st;
    gemm_norm_plan* p = new (std::nothrow) gemm_norm_plan();
    if (!p) return GEMM_ERR_OOM;
    p->max_rows = max_rows;
    p->cols = cols;
    p->elem = elem;
    p->weight_elem = weight_elem;
    p->device = device;
    p->num_sms = sms;
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
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        return gbt::launch(gbt::norm_forward_kernel<T, W>, rows, gbt::kThreads, 0, stream, 1,
                           static_cast<const T*>(x), ldx, static_cast<const W*>(gamma),
                           static_cast<const W*>(beta), eps, static_cast<T*>(y), ldy, mean, rstd,
                           static_cast<int>(p->cols));
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
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        gemm_status_t s = GEMM_OK;
        // (the weight's gradients first: dx may overwrite dy or x)
        if (dgamma || dbeta)
            s = gbt::launch(gbt::norm_weight_grad_kernel<T, W>, (p->cols + 31) / 32, gbt::kThreads,
                            0, stream, 1, static_cast<const T*>(x), ldx, mean, rstd,
                            static_cast<const T*>(dy), lddy, rows, static_cast<int>(p->cols),
                            static_cast<W*>(dgamma), static_cast<W*>(dbeta));
        if (s == GEMM_OK && dx && rows > 0)
            s = gbt::launch(gbt::norm_dx_kernel<T, W>, rows, gbt::kThreads, 0, stream, 1,
                            static_cast<const T*>(x), ldx, static_cast<const W*>(gamma), mean, rstd,
                            static_cast<const T*>(dy), lddy, static_cast<T*>(dx), lddx,
                            static_cast<int>(p->cols));
        return s;
    });
}

gemm_status_t gemm_norm_plan_destroy(gemm_norm_plan_t p) {
    delete p;
    return GEMM_OK;
}

}  // extern "C"
