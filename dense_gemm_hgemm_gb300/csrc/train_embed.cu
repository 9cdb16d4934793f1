// train_embed.cu -- embedding lookup of gemm_train.h and its table's gradient.
#include <new>

#include "train_common.cuh"

struct gemm_embed_plan {
    int64_t vocab, dim, max_tokens;
    gemm_elem_t elem, grad_elem;
    int device, num_sms;
    void* memory;            // one allocation: error word, sort buffers, partial sums
    int32_t* error_word;
    uint32_t* keys[2];
    uint32_t* pos[2];
    float* partial;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;

// ---- lookup ---------------------------------------------------------------------
//
// A group of `lanes` threads (a power of two, 8 to kThreads) takes TOKENS tokens: it loads
// their ids, then PACKS packs of each one's row in every thread, so that two chained loads
// serve TOKENS * PACKS * 16 bytes a thread.

struct LookupParams {
    const void* ids;
    int id_type;
    int64_t padding, tokens, vocab, ldt, ldo;
    float scale;
    int dim, lanes;
    int32_t* error;
};

// A pack times a number, or zeros.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> scaled(const Pack<T, VEC>& q, float scale, bool take) {
    Pack<T, VEC> r;
    if (!take) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.set_raw(i, from_f32<T>(0.f));
    } else if constexpr (VEC == 1) {
        r.set(0, scale * q.get(0));
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) set_pair(r, j, mul2(Pair(scale, scale), pair_of(q, j)));
    }
    return r;
}

template <typename T, int VEC, int PACKS, int TOKENS>
__global__ void __launch_bounds__(kThreads)
embed_forward_kernel(const LookupParams p, const T* __restrict__ table, T* __restrict__ out) {
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lane = threadIdx.x % p.lanes;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / p.lanes) + threadIdx.x / p.lanes) * TOKENS;
    int64_t id[TOKENS];
#pragma unroll
    for (int u = 0; u < TOKENS; ++u)
        id[u] = first + u < p.tokens ? load_index(p.ids, first + u, p.id_type) : p.padding;
#pragma unroll
    for (int u = 0; u < TOKENS; ++u) {
        if (id[u] == p.padding) {
            id[u] = -1;
        } else if (id[u] < 0 || id[u] >= p.vocab) {
            *p.error = kErrorIndex;
            id[u] = -1;
        }
    }
    for (int c0 = lane * VEC; c0 < p.dim; c0 += p.lanes * VEC * PACKS) {
        Pack<T, VEC> q[TOKENS][PACKS];
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
#pragma unroll
            for (int k = 0; k < PACKS; ++k) {
                const int c = c0 + k * p.lanes * VEC;
                if (id[u] >= 0 && c < p.dim) q[u][k] = load_pack<T, VEC>(table + id[u] * p.ldt + c, p.dim - c);
            }
        }
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            if (first + u >= p.tokens) return;
#pragma unroll
            for (int k = 0; k < PACKS; ++k) {
                const int c = c0 + k * p.lanes * VEC;
                if (c >= p.dim) break;
                store_pack<T, VEC>(out + (first + u) * p.ldo + c, p.dim - c, scaled(q[u][k], p.scale, id[u] >= 0));
            }
        }
    }
}

template <typename T, int VEC>
gemm_status_t lookup(LookupParams p, int sms, const T* table, T* out, void* stream) {
    constexpr int PACKS = 2;
    const int64_t packs = (static_cast<int64_t>(p.dim) + VEC - 1) / VEC;
    p.lanes = 8;
    while (p.lanes < kThreads && p.lanes * PACKS < packs) p.lanes *= 2;
    const int groups = kThreads / p.lanes;
    // four tokens a group where that leaves enough blocks to fill the GPU
    if (p.tokens >= int64_t{4} * 8 * sms * groups)
        return launch(embed_forward_kernel<T, VEC, PACKS, 4>, (p.tokens + 4 * groups - 1) / (4 * groups), kThreads,
                      0, stream, 1, p, table, out);
    return launch(embed_forward_kernel<T, VEC, PACKS, 1>, (p.tokens + groups - 1) / groups, kThreads, 0, stream, 1,
                  p, table, out);
}

// ---- the table's gradient -------------------------------------------------------
//
// The tokens are sorted by id (stable, so equal ids stay in the order of their
// positions), and sums go along the sorted order:
//   1. embed_sort_kernel: one thread-block cluster sorts (id, position) pairs; the
//      other blocks meanwhile write the zeros of all rows without a token, which
//      they find by marking the batch's ids in a bitmap of their own rows.
//   2. embed_sum_kernel: chunks of kChunk sorted entries.  A group of lanes keeps the
//      running sum of its columns in registers and writes a table row where the id
//      changes; a row whose entries cross a chunk's border leaves fp32 partial sums.
//   3. embed_join_kernel: adds the partial sums of such a row in the order of the
//      chunks.
// Every byte of dout is read once and every row of dtable written once; only rows
// with many tokens add partial sums (8 bytes per kChunk elements, mostly in L2).

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortItems = 8;                              // keys a thread holds
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxCluster = 8;
constexpr int kBitmapRows = 1 << 16;
constexpr int kChunk = 16;

struct SortParams {
    const void* ids;
    int id_type;
    int64_t padding;
    int64_t tokens;
    uint32_t vocab;          // also the key of tokens that take no part: they sort last
    int passes, digit_bits;
    uint32_t* keys[2];       // ping-pong; the last pass writes keys[0], pos[0]
    uint32_t* pos[2];
    int32_t* error;
    int fill_shift;          // log2 of the number of zero-filling blocks, or -1 = none
    void* table;
    int64_t row_bytes, stride_bytes;
    int vector_rows;         // table rows are 16-byte aligned
};

struct SortShared {
    uint32_t total[kDigits];                 // this block's keys of each digit (read by the cluster)
    uint32_t start[kDigits];                 // where the block's next key of a digit goes
    uint32_t scan[kSortWarps];
    uint16_t warp_count[kSortWarps][kDigits];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// A word of the same shared-memory variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t load_of_rank(const uint32_t* p, uint32_t rank) {
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t remote, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
    return v;
}

// A token's sort key; ids outside the table are reported.
__device__ __forceinline__ uint32_t key_of(const SortParams& p, int64_t t, bool report) {
    const int64_t id = load_index(p.ids, t, p.id_type);
    if (id == p.padding) return p.vocab;
    if (id >= 0 && id < static_cast<int64_t>(p.vocab)) return static_cast<uint32_t>(id);
    if (report) *p.error = kErrorIndex;
    return p.vocab;
}

// One stable pass of a radix sort over the cluster: each block ranks a contiguous
// span of the input, tile by tile; a warp ranks 32 keys at a time by matching their
// digits, so no order depends on timing.
__device__ void sort_pass(const SortParams& p, SortShared& sh, int pass, int64_t begin, int64_t end,
                          uint32_t rank, uint32_t ranks) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int shift = pass * p.digit_bits;
    const uint32_t mask = (1u << p.digit_bits) - 1u;
    const int to = (p.passes - 1 - pass) & 1;
    const uint32_t* in_keys = p.keys[to ^ 1];
    const uint32_t* in_pos = p.pos[to ^ 1];
    uint32_t key[kSortItems], at[kSortItems];
    uint16_t place[kSortItems];

    const auto rank_tile = [&](int64_t tile) {
        for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads)
            reinterpret_cast<uint32_t*>(sh.warp_count)[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t e = tile + (warp * kSortItems + i) * 32 + lane;
            key[i] = 0;
            at[i] = 0;
            if (e < end) {
                key[i] = pass == 0 ? key_of(p, e, true) : __ldcg(in_keys + e);
                at[i] = pass == 0 ? static_cast<uint32_t>(e) : __ldcg(in_pos + e);
            }
        }
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t e = tile + (warp * kSortItems + i) * 32 + lane;
            const uint32_t d = e < end ? (key[i] >> shift) & mask : kDigits;
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const unsigned before = same & ((1u << lane) - 1u);
            const uint32_t base = e < end ? sh.warp_count[warp][d] : 0;
            place[i] = static_cast<uint16_t>(base + __popc(before));
            __syncwarp();
            if (e < end && before == 0) sh.warp_count[warp][d] = static_cast<uint16_t>(base + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        uint32_t sum = 0;                    // thread d: digit d's count in each warp -> its start
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = sh.warp_count[w][tid];
            sh.warp_count[w][tid] = static_cast<uint16_t>(sum);
            sum += c;
        }
        __syncthreads();
        return sum;
    };

    // the block's count of each digit
    const bool one_tile = end - begin <= kSortTile;
    uint32_t count = 0;
    if (one_tile) {
        count = rank_tile(begin);
    } else {
        for (int64_t tile = begin; tile < end; tile += kSortTile) count += rank_tile(tile);
    }
    sh.total[tid] = count;
    cluster_barrier();
    // where they go: all smaller digits, then this digit's keys of the blocks before
    uint32_t all = 0, lower = 0;
    for (uint32_t r = 0; r < ranks; ++r) {
        const uint32_t c = load_of_rank(&sh.total[tid], r);
        if (r < rank) lower += c;
        all += c;
    }
    uint32_t sum = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sh.scan[warp] = sum;
    __syncthreads();
    uint32_t first = 0;
    for (int w = 0; w < warp; ++w) first += sh.scan[w];
    sh.start[tid] = first + sum - all + lower;
    __syncthreads();
    for (int64_t tile = begin; tile < end; tile += kSortTile) {
        const uint32_t tile_count = one_tile ? 0 : rank_tile(tile);
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t e = tile + (warp * kSortItems + i) * 32 + lane;
            if (e < end) {
                const uint32_t d = (key[i] >> shift) & mask;
                const uint32_t dst = sh.start[d] + sh.warp_count[warp][d] + place[i];
                __stcg(p.keys[to] + dst, key[i]);
                __stcg(p.pos[to] + dst, at[i]);
            }
        }
        __syncthreads();
        sh.start[tid] += tile_count;
    }
    cluster_barrier();   // the written keys are visible, and the totals have been read
}

// Zeros for every row without a token among the rows v with v % 2^shift == block.
__device__ void fill_untouched(const SortParams& p, uint32_t* bitmap, uint32_t block) {
    const uint32_t step = 1u << p.fill_shift;
    const uint32_t rows = block < p.vocab ? (p.vocab - block + step - 1) >> p.fill_shift : 0;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t r0 = 0; r0 < rows; r0 += kBitmapRows) {
        const uint32_t n = min(rows - r0, static_cast<uint32_t>(kBitmapRows));
        for (uint32_t i = threadIdx.x; i < (n + 31) / 32; i += kSortThreads) bitmap[i] = 0;
        __syncthreads();
        for (int64_t t = threadIdx.x; t < p.tokens; t += kSortThreads) {
            const uint32_t key = key_of(p, t, false);
            if (key < p.vocab && (key & (step - 1u)) == block) {
                const uint32_t r = key >> p.fill_shift;
                if (r >= r0 && r - r0 < n) atomicOr(&bitmap[(r - r0) / 32], 1u << ((r - r0) % 32));
            }
        }
        __syncthreads();
        for (uint32_t r = warp; r < n; r += kSortWarps) {
            if (bitmap[r / 32] >> (r % 32) & 1u) continue;
            uint8_t* row = static_cast<uint8_t*>(p.table) +
                           (static_cast<int64_t>(r0 + r) * step + block) * p.stride_bytes;
            int64_t done = 0;
            if (p.vector_rows) {
                done = p.row_bytes / 16 * 16;
                for (int64_t b = lane * 16; b < done; b += 32 * 16)
                    __stcs(reinterpret_cast<uint4*>(row + b), make_uint4(0u, 0u, 0u, 0u));
            }
            for (int64_t b = done + lane * 2; b < p.row_bytes; b += 32 * 2)   // elements are 2 or 4 bytes
                *reinterpret_cast<uint16_t*>(row + b) = 0;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortParams p, int ranks) {
    __shared__ union {
        SortShared sort;
        uint32_t bitmap[kBitmapRows / 32];
    } sh;
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (blockIdx.x >= static_cast<unsigned>(ranks)) {
        fill_untouched(p, sh.bitmap, blockIdx.x - ranks);
        return;
    }
    const uint32_t rank = cluster_rank();
    const int64_t per = ((p.tokens + ranks - 1) / ranks + 31) / 32 * 32;
    const int64_t begin = min(p.tokens, rank * per), end = min(p.tokens, begin + per);
    for (int pass = 0; pass < p.passes; ++pass) sort_pass(p, sh.sort, pass, begin, end, rank, ranks);
}

struct SumParams {
    const uint32_t* keys;
    const uint32_t* pos;
    uint32_t vocab;
    int64_t tokens, chunks;
    int dim, lanes, col_tiles;   // lanes: of a group, a power of two
    int64_t ldo, ldt;
    float scale;
    int accumulate;
    float* partial;              // [2][chunks][dim]: what a chunk adds to a row that begins
                                 // before it (0), and to one that goes on behind it (1)
};

template <typename G, int VEC>
__device__ __forceinline__ void write_row(const SumParams& p, G* table, uint32_t key, int64_t c,
                                          const float (&sum)[VEC], const float (&old)[VEC]) {
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p.accumulate ? old[i] + p.scale * sum[i] : p.scale * sum[i];
    store_values<G, VEC>(table + key * p.ldt + c, p.dim - c, v);
}

template <typename T, typename G, int VEC>
__global__ void __launch_bounds__(kThreads)
embed_sum_kernel(const SumParams p, const T* __restrict__ dout, G* __restrict__ table) {
    constexpr int kAhead = 8;
    static_assert(kChunk % kAhead == 0, "whole batches of rows");
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int groups = kThreads / p.lanes;
    const int64_t chunk = static_cast<int64_t>(blockIdx.x) / p.col_tiles * groups + threadIdx.x / p.lanes;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % p.col_tiles) * p.lanes + threadIdx.x % p.lanes) * VEC;
    if (chunk >= p.chunks || c >= p.dim) return;
    const int64_t first = chunk * kChunk;
    bool began_before = first > 0 && p.keys[first - 1] == p.keys[first];
    float sum[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
    for (int b = 0; b < kChunk; b += kAhead) {
        uint32_t key[kAhead + 1];
        Pack<T, VEC> row[kAhead];
#pragma unroll
        for (int u = 0; u <= kAhead; ++u)
            key[u] = first + b + u < p.tokens ? p.keys[first + b + u] : p.vocab;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (key[u] < p.vocab)
                row[u] = load_pack<T, VEC>(dout + p.pos[first + b + u] * p.ldo + c, p.dim - c);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (key[u] >= p.vocab) return;       // the rest takes no part
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] += row[u].get(i);
            const bool last = b + u == kChunk - 1;
            if (key[u + 1] == key[u] && !last) continue;
            if (key[u + 1] == key[u] || began_before) {
                float* at = p.partial + ((began_before ? 0 : p.chunks) + chunk) * p.dim + c;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i < p.dim) at[i] = sum[i];
            } else {
                float old[VEC];
                if (p.accumulate) load_values<G, VEC>(table + key[u] * p.ldt + c, p.dim - c, old);
                write_row<G, VEC>(p, table, key[u], c, sum, old);
            }
            began_before = false;
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
        }
    }
}

// One block per chunk and 32 columns x VEC: if a row begins in the chunk and goes on
// behind it, its warps take the partial sums of the following chunks in turn.
template <typename G, int VEC>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const SumParams p, G* __restrict__ table) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float part[kWarps][32][VEC + 1];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int tiles = (p.dim + 32 * VEC - 1) / (32 * VEC);
    const int64_t chunk = static_cast<int64_t>(blockIdx.x) / tiles;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % tiles) * 32 + lane) * VEC;
    const int64_t first = chunk * kChunk, next = first + kChunk;
    const uint32_t key = p.keys[next - 1];        // (chunks that end inside the tokens only)
    if (key >= p.vocab || p.keys[next] != key || (first > 0 && p.keys[first - 1] == key)) return;
    float sum[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
    const auto add = [&](const float* at) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < p.dim) sum[i] += at[c + i];
    };
    if (warp == 0) add(p.partial + (p.chunks + chunk) * p.dim);
    for (int64_t k = chunk + 1 + warp; k * kChunk < p.tokens && p.keys[k * kChunk] == key; k += kWarps)
        add(p.partial + k * p.dim);
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[warp][lane][i] = sum[i];
    __syncthreads();
    if (warp != 0 || c >= p.dim) return;
    for (int w = 1; w < kWarps; ++w) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += part[w][lane][i];
    }
    float old[VEC];
    if (p.accumulate) load_values<G, VEC>(table + key * p.ldt + c, p.dim - c, old);
    write_row<G, VEC>(p, table, key, c, sum, old);
}

int64_t chunks_of(int64_t tokens) { return (tokens + kChunk - 1) / kChunk; }

template <typename T, typename G, int VEC>
gemm_status_t sum_rows(SumParams s, const T* dout, G* table, void* stream) {
    const int64_t packs = (s.dim + VEC - 1) / VEC;
    s.lanes = 8;
    while (s.lanes < kThreads && s.lanes < packs) s.lanes *= 2;
    s.col_tiles = static_cast<int>((packs + s.lanes - 1) / s.lanes);
    const int groups = kThreads / s.lanes;
    const gemm_status_t st =
        launch(embed_sum_kernel<T, G, VEC>, (s.chunks + groups - 1) / groups * s.col_tiles, kThreads, 0,
               stream, 1, s, dout, table);
    const int64_t crossings = (s.tokens - 1) / kChunk;      // chunks with a token behind them
    if (st != GEMM_OK || crossings == 0) return st;
    return launch(embed_join_kernel<G, VEC>, crossings * ((s.dim + 32 * VEC - 1) / (32 * VEC)), kThreads,
                  0, stream, 1, s, table);
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
    const auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
    const size_t list = padded(static_cast<size_t>(max_tokens) * 4);
    const size_t sums = static_cast<size_t>(gbt::chunks_of(max_tokens)) * 2 * static_cast<size_t>(dim) * 4;
    void* memory = nullptr;
    st = gbt::allocate(&memory, 256 + 4 * list + sums);
    if (st != GEMM_OK) return st;
    gemm_embed_plan* p = new (std::nothrow) gemm_embed_plan();
    if (!p || cudaMemset(memory, 0, 256) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(memory);
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
    p->memory = memory;
    p->error_word = static_cast<int32_t*>(memory);
    uint8_t* at = static_cast<uint8_t*>(memory) + 256;
    for (int k = 0; k < 2; ++k, at += 2 * list) {
        p->keys[k] = reinterpret_cast<uint32_t*>(at);
        p->pos[k] = reinterpret_cast<uint32_t*>(at + list);
    }
    p->partial = reinterpret_cast<float*>(at);
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
    const gbt::LookupParams q{ids,  static_cast<int>(id_type), padding, tokens, p->vocab, ldt, ldo, scale,
                              static_cast<int>(p->dim), 0, p->error_word};
    const bool vec = gbt::rows_aligned(table, ldt, e) && gbt::rows_aligned(out, ldo, e);
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        const T* from = static_cast<const T*>(table);
        T* to = static_cast<T*>(out);
        return vec ? gbt::lookup<T, kVec>(q, p->num_sms, from, to, stream)
                   : gbt::lookup<T, 1>(q, p->num_sms, from, to, stream);
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
    gemm_status_t st = gbt::check_device(p->device);
    if (st != GEMM_OK || (tokens == 0 && accumulate)) return st;
    const int g = gbt::elem_bytes(p->grad_elem);

    gbt::SortParams q = {};
    q.ids = ids;
    q.id_type = static_cast<int>(id_type);
    q.padding = padding;
    q.tokens = tokens;
    q.vocab = static_cast<uint32_t>(p->vocab);
    int bits = 1;
    while (p->vocab >> bits != 0) ++bits;      // keys up to vocab itself
    q.passes = (bits + gbt::kDigitBits - 1) / gbt::kDigitBits;
    q.digit_bits = (bits + q.passes - 1) / q.passes;
    for (int k = 0; k < 2; ++k) {
        q.keys[k] = p->keys[k];
        q.pos[k] = p->pos[k];
    }
    q.error = p->error_word;
    q.fill_shift = -1;
    q.table = dtable;
    q.row_bytes = p->dim * g;
    q.stride_bytes = ldt * g;
    q.vector_rows = gbt::rows_aligned(dtable, ldt, g);
    // the sorting cluster: about 512 tokens a block
    int ranks = 1;
    while (ranks < gbt::kMaxCluster && ranks * 512 < tokens) ranks *= 2;
    int64_t grid = ranks;
    if (!accumulate) {
        // zero-filling blocks: a power of two (a row's block is in its id's low bits), whole
        // clusters, at least 64 KiB each
        q.fill_shift = 0;
        while ((1 << q.fill_shift) < ranks ||
               (q.fill_shift < 9 && (p->vocab * q.row_bytes) >> (16 + q.fill_shift) != 0))
            ++q.fill_shift;
        grid += int64_t{1} << q.fill_shift;
    }
    st = gbt::launch(gbt::embed_sort_kernel, grid, gbt::kSortThreads, 0, stream, ranks, q, ranks);
    if (st != GEMM_OK || tokens == 0) return st;

    gbt::SumParams s = {};
    s.keys = p->keys[0];
    s.pos = p->pos[0];
    s.vocab = q.vocab;
    s.tokens = tokens;
    s.chunks = gbt::chunks_of(tokens);
    s.dim = static_cast<int>(p->dim);
    s.ldo = ldo;
    s.ldt = ldt;
    s.scale = scale;
    s.accumulate = accumulate;
    s.partial = p->partial;
    const int e = gbt::elem_bytes(p->elem);
    const bool vec = gbt::rows_aligned(dout, ldo, e) && q.vector_rows;
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        const auto run = [&](auto v) {
            using G = decltype(v);
            const T* d = static_cast<const T*>(dout);
            G* w = static_cast<G*>(dtable);
            return vec ? gbt::sum_rows<T, G, kVec>(s, d, w, stream) : gbt::sum_rows<T, G, 1>(s, d, w, stream);
        };
        return p->grad_elem == GEMM_ELEM_F32 ? run(float()) : run(t);
    });
}

gemm_status_t gemm_embed_plan_check(gemm_embed_plan_t p, void* stream) {
    return p ? gbt::check_error_word(p->error_word, stream) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_embed_plan_destroy(gemm_embed_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = cudaFree(p->memory) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    if (st != GEMM_OK) cudaGetLastError();
    delete p;
    return st;
}

}  // extern "C"
