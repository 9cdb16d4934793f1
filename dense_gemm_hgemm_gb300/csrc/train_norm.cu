// train_norm.cu -- layer norm of gemm_train.h, forward and backward.
#include <new>

#include "train_common.cuh"

struct gemm_norm_plan {
    int64_t max_rows, cols;
    gemm_elem_t elem, weight_elem;
    int device, num_sms;
    float* partial;      // [2][blocks][cols] sums of the weight gradients
};

namespace gbt {
namespace {

constexpr int kThreads = 256;      // of the kernels that loop over a row or a column
constexpr int kMaxLanes = 1024;
constexpr int kLaneCols = 16;      // columns a lane keeps in registers

// ---- rows in registers ----------------------------------------------------------
//
// `lanes` threads (32 to 1024, a power of two) keep one row, kLaneCols columns each:
// PACKS packs of VEC elements, pack k of lane l at column (k * lanes + l) * VEC.  A
// block has BLOCK / lanes such groups, each with its own rows, and asks for its next
// row before it works on the present one.  So a row is read once, and its statistics
// are exact two-pass ones at no further traffic.

template <typename T, int VEC>
struct RowPacks {
    static constexpr int PACKS = kLaneCols / VEC;
    Pack<T, VEC> p[PACKS];
    __device__ __forceinline__ void load(const T* row, int lane, int lanes, int cols) {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = (k * lanes + lane) * VEC;
            p[k] = load_pack<T, VEC>(row + c, cols - c);
        }
    }
    __device__ __forceinline__ void store(T* row, int lane, int lanes, int cols) const {
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            const int c = (k * lanes + lane) * VEC;
            store_pack<T, VEC>(row + c, cols - c, p[k]);
        }
    }
};

constexpr int kPairs = kLaneCols / 2;

// A lane's columns of a weight vector (`other` without one, and past the row's end).
template <typename W, int VEC>
__device__ __forceinline__ void load_weights(const W* w, float other, int lane, int lanes, int cols, Pair (&v)[kPairs]) {
    constexpr int PACKS = kLaneCols / VEC;
    float f[kLaneCols];
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
        const int c = (k * lanes + lane) * VEC;
        float part[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) part[i] = other;
        if (w) load_values<W, VEC>(w + c, cols - c, part);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[k * VEC + i] = part[i];
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) v[j] = Pair(f[2 * j], f[2 * j + 1]);
}

__device__ __forceinline__ float sum_of(const Pair (&v)[kPairs]) {
    Pair s = add2(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < kPairs; ++j) s = add2(s, v[j]);
    float lo, hi;
    s.get(lo, hi);
    return lo + hi;
}

// Sums over a group, in every lane: shuffles in the warp, then one exchange in shared
// memory behind the group's own barrier.  Two exchange buffers in turn: a warp that is
// a sum ahead has passed the barrier that the others reach only after their reads.
template <int N>
struct GroupSum {
    float (*part)[N][32];    // [2][N][32] of the group
    int lanes, barrier, turn;
    __device__ __forceinline__ void operator()(float (&v)[N], int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (lanes == 32) return;
        const int warps = lanes / 32, l = lane % 32;
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) part[turn][i][lane / 32] = v[i];
        }
        asm volatile("bar.sync %0, %1;" :: "r"(barrier), "r"(lanes) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(l < warps ? part[turn][i][l] : 0.f);
        turn ^= 1;
    }
};

template <typename T, typename W>
struct ForwardArgs {
    const T* x;
    const W* gamma;
    const W* beta;
    T* y;
    float* mean;
    float* rstd;
    int64_t ldx, ldy, rows;
    float eps;
    int cols, lanes;
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
    GroupSum<1> sum{part[group], lanes, 1 + group, 0};
    RowPacks<T, VEC> next;
    next.load(a.x + row * a.ldx, lane, lanes, a.cols);
    Pair gamma[kPairs], beta[kPairs];
    if (KEEP) {
        load_weights<W, VEC>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
        load_weights<W, VEC>(a.beta, 0.f, lane, lanes, a.cols, beta);
    }
    const float n = static_cast<float>(a.cols);
    for (; row < a.rows; row += step) {
        Pair v[kPairs];
        to_pairs(next.p, v);                     // (columns past the row's end are zeros)
        if (row + step < a.rows) next.load(a.x + (row + step) * a.ldx, lane, lanes, a.cols);
        float s[1] = {sum_of(v)};
        sum(s, lane);
        const float mu = s[0] / n;
        const Pair minus(-mu, -mu);
        Pair square(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = add2(v[j], minus);
        if (!full) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const int k = 2 * j / VEC, c = (k * lanes + lane) * VEC + 2 * j % VEC;
                const int c1 = VEC == 1 ? c + lanes : c + 1;
                float lo, hi;
                v[j].get(lo, hi);
                v[j] = Pair(c < a.cols ? lo : 0.f, c1 < a.cols ? hi : 0.f);
            }
        }
#pragma unroll
        for (int j = 0; j < kPairs; ++j) square = fma2(v[j], v[j], square);
        float lo, hi;
        square.get(lo, hi);
        s[0] = lo + hi;
        sum(s, lane);
        const float r = 1.f / sqrtf(s[0] / n + a.eps);
        if (!KEEP) {
            load_weights<W, VEC>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
            load_weights<W, VEC>(a.beta, 0.f, lane, lanes, a.cols, beta);
        }
        const Pair r2(r, r);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) v[j] = fma2(mul2(v[j], r2), gamma[j], beta[j]);
        RowPacks<T, VEC> out;
        from_pairs(v, out.p);
        out.store(a.y + row * a.ldy, lane, lanes, a.cols);
        if (lane == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
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
    int64_t ldx, lddy, lddx, rows;
    int cols, lanes;
    bool weights;        // dgamma or dbeta is wanted
};

// dx of each row, and the block's sums of dy * xh and dy over its rows: each lane adds
// up its own columns, in registers (SHARED: in shared memory, where a block of 1024
// threads has no registers left for them); the groups of a block are joined at the end.
template <typename T, typename W, int VEC, int BLOCK, bool SHARED>
__global__ void __launch_bounds__(BLOCK) norm_backward_kernel(const BackwardArgs<T, W> a) {
    extern __shared__ float join[];      // [2][lanes * kLaneCols]
    __shared__ float part[BLOCK / 32][2][2][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lanes = a.lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int groups = BLOCK / lanes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
    GroupSum<2> sum{part[group], lanes, 1 + group, 0};
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
    if (!SHARED) load_weights<W, VEC>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
    RowPacks<T, VEC> next_x, next_dy;
    float next_mean = 0.f, next_rstd = 0.f;
    const auto ask = [&](int64_t r) {
        next_x.load(a.x + r * a.ldx, lane, lanes, a.cols);
        next_dy.load(a.dy + r * a.lddy, lane, lanes, a.cols);
        next_mean = a.mean[r];
        next_rstd = a.rstd[r];
    };
    if (row < a.rows) ask(row);
    const float n = static_cast<float>(a.cols);
    for (; row < a.rows; row += step) {
        const float mu = next_mean, r = next_rstd;
        Pair hat[kPairs], g[kPairs];
        to_pairs(next_x.p, hat);
        to_pairs(next_dy.p, g);                  // dy: zero past the row's end, as every sum's term there
        if (row + step < a.rows) ask(row + step);
        if (SHARED) load_weights<W, VEC>(a.gamma, 1.f, lane, lanes, a.cols, gamma);
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
        float lo, hi, s[2];
        sum_g.get(lo, hi);
        s[0] = lo + hi;
        sum_gx.get(lo, hi);
        s[1] = lo + hi;
        sum(s, lane);
        const float mean_g = s[0] / n, mean_gx = s[1] / n;
        const Pair minus_g(-mean_g, -mean_g), minus_gx(-mean_gx, -mean_gx);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) g[j] = mul2(r2, fma2(hat[j], minus_gx, add2(g[j], minus_g)));
        RowPacks<T, VEC> out;
        from_pairs(g, out.p);
        out.store(a.dx + row * a.lddx, lane, lanes, a.cols);
    }
    if (!a.weights) return;
    if (!SHARED) {
        for (int turn = 0; turn < groups; ++turn) {      // the groups in turn
            if (group == turn) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    add_to(0, j, dg[j], turn == 0);
                    add_to(1, j, db[j], turn == 0);
                }
            }
            __syncthreads();
        }
    } else {
        __syncthreads();
    }
    for (int which = 0; which < 2; ++which) {
        float* out = a.partial + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.cols;
        for (int c = threadIdx.x; c < a.cols; c += BLOCK) {
            const int pack = c / VEC;            // column c is element c % VEC of this pack
            out[c] = join[(which * kLaneCols + pack / lanes * VEC + c % VEC) * lanes + pack % lanes];
        }
    }
}

// The blocks' sums of 32 columns: eight warps take every eighth block, then join.
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
    if (c < cols)
        for (int b = warp; b < blocks; b += kThreads / 32)
            s += partial[(static_cast<int64_t>(which) * blocks + b) * cols + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= cols) return;
    for (int w = 1; w < kThreads / 32; ++w) s += part[w][lane];
    out[c] = from_f32<W>(s);
}

// ---- rows too wide for the registers of a block ------------------------------------

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

// Lanes that keep a row of `cols` columns.
int lanes_for(int64_t cols) {
    int lanes = 32;
    while (static_cast<int64_t>(lanes) * kLaneCols < cols) lanes *= 2;
    return lanes;
}

bool in_registers(int64_t cols) { return cols <= static_cast<int64_t>(kMaxLanes) * kLaneCols; }

template <typename T, typename W, int VEC, int BLOCK, bool KEEP>
gemm_status_t forward_rows(const ForwardArgs<T, W>& a, int sms, void* stream) {
    const auto kernel = norm_forward_kernel<T, W, VEC, BLOCK, KEEP>;
    const int groups = BLOCK / a.lanes;
    const int64_t blocks = (a.rows + groups - 1) / groups;
    const int64_t most = static_cast<int64_t>(sms) * (2048 / BLOCK);
    return launch(kernel, blocks < most ? blocks : most, BLOCK, 0, stream, 1, a);
}

template <typename T, typename W, int VEC>
gemm_status_t forward_vec(const ForwardArgs<T, W>& a, int sms, void* stream) {
    if (a.lanes <= 256) return forward_rows<T, W, VEC, 256, true>(a, sms, stream);
    if (a.lanes == 512) return forward_rows<T, W, VEC, 512, true>(a, sms, stream);
    return forward_rows<T, W, VEC, 1024, false>(a, sms, stream);
}

template <typename T, typename W, int VEC, int BLOCK, bool SHARED>
gemm_status_t backward_rows(const BackwardArgs<T, W>& a, int blocks, void* stream) {
    const auto kernel = norm_backward_kernel<T, W, VEC, BLOCK, SHARED>;
    // (SHARED keeps its sums there whether they are wanted or not)
    const size_t smem = SHARED || a.weights ? static_cast<size_t>(a.lanes) * kLaneCols * 2 * sizeof(float) : 0;
    return launch(kernel, blocks, BLOCK, smem, stream, 1, a);
}

// Lets the kernels have as much shared memory as their largest launch asks for.
template <typename T, typename W>
gemm_status_t prepare() {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const auto allow = [](auto kernel, int lanes) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    lanes * kLaneCols * 2 * static_cast<int>(sizeof(float))) == cudaSuccess;
    };
    if (allow(norm_backward_kernel<T, W, kVec, 512, false>, 512) && allow(norm_backward_kernel<T, W, 1, 512, false>, 512) &&
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

template <typename T, typename W, int VEC>
gemm_status_t backward_vec(const BackwardArgs<T, W>& a, int blocks, void* stream) {
    if (a.lanes <= 512) return backward_rows<T, W, VEC, 512, false>(a, blocks, stream);
    return backward_rows<T, W, VEC, 1024, true>(a, blocks, stream);
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
    void* partial = nullptr;
    if (max_rows > 0 && gbt::in_registers(cols)) {
        const int64_t blocks = gbt::backward_blocks(max_rows, gbt::lanes_for(cols), sms);
        const gemm_status_t room = gbt::allocate(&partial, static_cast<size_t>(blocks * cols) * 2 * sizeof(float));
        if (room != GEMM_OK) return room;
    }
    gemm_norm_plan* p = new (std::nothrow) gemm_norm_plan();
    if (!p) {
        cudaFree(partial);
        return GEMM_ERR_OOM;
    }
    p->max_rows = max_rows;
    p->cols = cols;
    p->elem = elem;
    p->weight_elem = weight_elem;
    p->device = device;
    p->num_sms = sms;
    p->partial = static_cast<float*>(partial);
    const gemm_status_t ready =
        gbt::with_types(p, [](auto t, auto v) { return gbt::prepare<decltype(t), decltype(v)>(); });
    if (ready != GEMM_OK) {
        cudaFree(partial);
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
    return gbt::with_types(p, [&](auto t, auto v) {
        using T = decltype(t);
        using W = decltype(v);
        const gbt::ForwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const W*>(gamma),
                                       static_cast<const W*>(beta), static_cast<T*>(y), mean, rstd,
                                       ldx, ldy, rows, eps, static_cast<int>(p->cols),
                                       gbt::lanes_for(p->cols)};
        if (!gbt::in_registers(p->cols))
            return gbt::launch(gbt::norm_forward_wide_kernel<T, W>, rows, gbt::kThreads, 0, stream, 1, a);
        const bool vec = gbt::rows_aligned(x, ldx, e) && gbt::rows_aligned(y, ldy, e) &&
                         gbt::aligned(gamma, 16) && gbt::aligned(beta, 16);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        return vec ? gbt::forward_vec<T, W, kVec>(a, p->num_sms, stream)
                   : gbt::forward_vec<T, W, 1>(a, p->num_sms, stream);
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
        W* dg = static_cast<W*>(dgamma);
        W* db = static_cast<W*>(dbeta);
        const int lanes = gbt::lanes_for(p->cols);
        gbt::BackwardArgs<T, W> a{static_cast<const T*>(x), static_cast<const W*>(gamma), mean, rstd,
                                  static_cast<const T*>(dy), static_cast<T*>(dx), p->partial, ldx,
                                  lddy, lddx, rows, static_cast<int>(p->cols), lanes, dg || db};
        const int tiles = static_cast<int>((p->cols + 31) / 32);
        gemm_status_t s = GEMM_OK;
        if (!gbt::in_registers(p->cols)) {
            // (the weight's gradients first: dx may overwrite dy or x)
            if (a.weights)
                s = gbt::launch(gbt::norm_weight_grad_wide_kernel<T, W>, tiles, gbt::kThreads, 0, stream,
                                1, a, dg, db);
            if (s == GEMM_OK && dx && rows > 0)
                s = gbt::launch(gbt::norm_dx_wide_kernel<T, W>, rows, gbt::kThreads, 0, stream, 1, a);
            return s;
        }
        const int blocks = static_cast<int>(gbt::backward_blocks(rows, lanes, p->num_sms));
        if (blocks > 0) {
            const bool vec = gbt::rows_aligned(x, ldx, e) && gbt::rows_aligned(dy, lddy, e) &&
                             (!dx || gbt::rows_aligned(dx, lddx, e)) && gbt::aligned(gamma, 16);
            constexpr int kVec = 16 / static_cast<int>(sizeof(T));
            s = vec ? gbt::backward_vec<T, W, kVec>(a, blocks, stream)
                    : gbt::backward_vec<T, W, 1>(a, blocks, stream);
        }
        if (s == GEMM_OK && a.weights)
            s = gbt::launch(gbt::norm_weight_join_kernel<W>, 2 * tiles, gbt::kThreads, 0, stream, 1,
                            p->partial, blocks, static_cast<int>(p->cols), dg, db);
        return s;
    });
}

gemm_status_t gemm_norm_plan_destroy(gemm_norm_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->partial) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
