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
    uint32_t* long_rows;
    float* partial;
};

namespace gbt {
namespace {

constexpr int kThreads = 256;

// ---- lookup ---------------------------------------------------------------------
//
// Bound by bytes: each token's row read (in L2 for frequent tokens) and written.  A group of
// `lanes` threads (a power of two, 8 to kThreads) takes TOKENS tokens: it loads their ids,
// then PACKS packs of each one's row in every thread, so that two chained loads serve
// TOKENS * PACKS * 16 bytes a thread.  16384 tokens of 128000 x 4096 bf16: 32.2 us, 5.9 TB/s
// of what has to move, with four tokens and one pack at a time; 35.7 us with two packs, 33.9
// with one token and two packs, 70 us where the elements were converted one by one.

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
            if (first + u >= p.tokens) break;            // (the tokens before go on with further columns)
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
gemm_status_t lookup(LookupParams p, int sms, const T* table, T* out, Queue queue) {
    constexpr int PACKS = 2;
    const int64_t packs = (static_cast<int64_t>(p.dim) + VEC - 1) / VEC;
    p.lanes = 8;
    while (p.lanes < kThreads && p.lanes * PACKS < packs) p.lanes *= 2;
    const int groups = kThreads / p.lanes;
    // four tokens a group where that leaves enough blocks to fill the GPU (with fewer tokens
    // the first loads' latency counts: 8 tokens 1.9 us)
    if (p.tokens >= int64_t{4} * 8 * sms * groups)
        return launch<embed_forward_kernel<T, VEC, 1, 4>>((p.tokens + 4 * groups - 1) / (4 * groups), kThreads,
                      0, queue, 1, p, table, out);
    return launch<embed_forward_kernel<T, VEC, PACKS, 1>>((p.tokens + groups - 1) / groups, kThreads, 0, queue, 1,
                  p, table, out);
}

// ---- the table's gradient -------------------------------------------------------
//
// The tokens are sorted by id (stable, so equal ids stay in the order of their
// positions), and sums go along the sorted order:
//   1. embed_sort_kernel: one thread-block cluster sorts (id, position) pairs; the
//      other blocks meanwhile write the zeros of all rows without a token, which
//      they find by marking the batch's ids in a bitmap of their own rows.
//   2. embed_sum_kernel: the sorted entries are cut into chunks.  A warp keeps the
//      running sum of its columns in registers and writes a table row where the id
//      changes.  A row with at most a chunk's entries is summed whole by the chunk
//      that it begins in; a longer one leaves an fp32 partial sum per chunk.
//   3. embed_join_kernel: adds the partial sums of each longer row in the order of
//      the chunks.
// Every byte of dout is read once and every row of dtable written once; only rows with
// more than a chunk of tokens add partial sums (8 bytes per element and chunk, in L2).  The
// sums of a row are added in the order of its tokens, chunk by chunk: no order depends on
// timing.
//
// Bound, and measured: 16384 tokens into 64000 x 4096 bf16 written whole take 131 us against
// 98 for the bytes: 80 to write 477 MB of zeros (5.9 TB/s: the store path, not the sort
// beside it, which is done by then), 35 to sum, 5 to join.  Writing the zeros by bulk stores
// from shared memory was not faster.  4099 tokens added to 50021 x 1000 fp32 take 18 us: 9, 6
// and 3 us of latency (loads that wait on one another, cluster barriers) against 3.5 for the
// bytes.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortItems = 4;                              // keys a thread holds
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxCluster = 8;
constexpr int kSortBlock = 1024;
constexpr int kBitmapRows = 1 << 16;

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
    uint32_t* long_rows;     // count of the rows with partial sums: cleared here
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
    uint2 pairs[kSortTile];                  // (key, position) between passes, where a block's keys are one tile
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

// A pair into the same variable of block `rank`.
__device__ __forceinline__ void store_to_rank(uint2* p, uint32_t rank, uint32_t x, uint32_t y) {
    const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" :: "r"(remote), "r"(x), "r"(y) : "memory");
}

// A token's sort key; ids outside the table are reported.
__device__ __forceinline__ uint32_t key_of(const SortParams& p, int64_t t, bool report) {
    const int64_t id = load_index(p.ids, t, p.id_type);
    if (id == p.padding) return p.vocab;
    if (id >= 0 && id < static_cast<int64_t>(p.vocab)) return static_cast<uint32_t>(id);
    if (report) *p.error = kErrorIndex;
    return p.vocab;
}

// One cluster, as its blocks must meet between passes: up to 16384 tokens have their pairs in
// its shared memory throughout (with the passes through global memory, and partial sums for
// every row that crosses a chunk, the 4099 tokens above took 28 us).  Digits of up to 9 bits,
// one thread each: two passes serve up to 2^18 - 1 rows (the number of rows is a key itself).
// More tokens go through global memory, each ranked twice a pass: 32768 into 64000 x 1024 bf16
// written whole take 82 us against 29 for the bytes, 131072 take 234 against 59.
//
// One stable pass of a radix sort over the cluster: each block ranks a contiguous span of
// the input, tile by tile; a warp ranks 32 keys at a time by matching their digits, so no
// order depends on timing.  Where each block has one tile, the pairs go from pass to pass
// through the cluster's shared memory (else through global memory).
__device__ void sort_pass(const SortParams& p, SortShared& sh, int pass, int64_t per, int64_t begin, int64_t end,
                          uint32_t rank, uint32_t ranks) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int shift = pass * p.digit_bits;
    const uint32_t mask = (1u << p.digit_bits) - 1u;
    const int to = (p.passes - 1 - pass) & 1;
    const bool one_tile = per <= kSortTile;
    const int items = static_cast<int>(min(per, static_cast<int64_t>(kSortTile)) + kSortThreads - 1) / kSortThreads;
    uint32_t key[kSortItems], at[kSortItems];
    uint16_t place[kSortItems];

    const auto entry = [&](int64_t tile, int i) { return tile + (warp * items + i) * 32 + lane; };
    const auto rank_tile = [&](int64_t tile) {
        for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads)
            reinterpret_cast<uint32_t*>(sh.warp_count)[i] = 0;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            const int64_t e = entry(tile, i);
            key[i] = 0;
            at[i] = 0;
            if (i < items && e < end) {
                if (pass == 0) {
                    key[i] = key_of(p, e, true);
                    at[i] = static_cast<uint32_t>(e);
                } else if (one_tile) {
                    const uint2 v = sh.pairs[e - begin];
                    key[i] = v.x;
                    at[i] = v.y;
                } else {
                    key[i] = __ldcg(p.keys[to ^ 1] + e);
                    at[i] = __ldcg(p.pos[to ^ 1] + e);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            if (i >= items) break;
            const bool valid = entry(tile, i) < end;
            const uint32_t d = valid ? (key[i] >> shift) & mask : kDigits;
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const unsigned before = same & ((1u << lane) - 1u);
            const uint32_t base = valid ? sh.warp_count[warp][d] : 0;
            place[i] = static_cast<uint16_t>(base + __popc(before));
            __syncwarp();
            if (valid && before == 0) sh.warp_count[warp][d] = static_cast<uint16_t>(base + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        uint32_t sum = 0;                    // thread d: digit d's count in each warp -> its start
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = sh.warp_count[w][tid];
            sh.warp_count[w][tid] = static_cast<uint16_t>(sum);
            sum += c;
        }
        return sum;
    };

    // the block's count of each digit
    uint32_t count = 0;
    if (one_tile) {
        count = rank_tile(begin);
    } else {
        for (int64_t tile = begin; tile < end; tile += kSortTile) {
            count += rank_tile(tile);
            __syncthreads();
        }
    }
    sh.total[tid] = count;
    uint32_t all = count, lower = 0;
    if (ranks > 1) {
        cluster_barrier();                   // (and all pairs of the pass before have been read)
        // where they go: all smaller digits, then this digit's keys of the blocks before
        all = 0;
        uint32_t c[kMaxCluster];
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) c[r] = r < ranks ? load_of_rank(&sh.total[tid], r) : 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            if (r < rank) lower += c[r];
            all += c[r];
        }
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
    const bool last = pass == p.passes - 1;
    for (int64_t tile = begin; tile < end; tile += kSortTile) {
        const uint32_t tile_count = one_tile ? 0 : rank_tile(tile);
        if (!one_tile) __syncthreads();
#pragma unroll
        for (int i = 0; i < kSortItems; ++i) {
            if (i >= items || entry(tile, i) >= end) break;
            const uint32_t d = (key[i] >> shift) & mask;
            const uint32_t dst = sh.start[d] + sh.warp_count[warp][d] + place[i];
            if (one_tile && !last) {
                const uint32_t owner = dst / static_cast<uint32_t>(per);
                store_to_rank(&sh.pairs[dst - owner * static_cast<uint32_t>(per)], owner, key[i], at[i]);
            } else {
                __stcg(p.keys[to] + dst, key[i]);
                __stcg(p.pos[to] + dst, at[i]);
            }
        }
        __syncthreads();
        sh.start[tid] += tile_count;
    }
    if (ranks > 1) cluster_barrier();        // what was written is visible, and the totals have been read
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
        constexpr int kAhead = 8;                // ids in flight a thread
        for (int64_t t0 = threadIdx.x; t0 < p.tokens; t0 += kAhead * kSortThreads) {
            uint32_t key[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                key[u] = t0 + u * kSortThreads < p.tokens ? key_of(p, t0 + u * kSortThreads, false) : p.vocab;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (key[u] >= p.vocab || (key[u] & (step - 1u)) != block) continue;
                const uint32_t r = key[u] >> p.fill_shift;
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
    extern __shared__ __align__(16) uint8_t memory[];    // SortShared, or a bitmap of kBitmapRows
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (blockIdx.x >= static_cast<unsigned>(ranks)) {
        fill_untouched(p, reinterpret_cast<uint32_t*>(memory), blockIdx.x - ranks);
        return;
    }
    SortShared& sh = *reinterpret_cast<SortShared*>(memory);
    const uint32_t rank = cluster_rank();
    if (rank == 0 && threadIdx.x == 0) *p.long_rows = 0;
    const int64_t per = ((p.tokens + ranks - 1) / ranks + 31) / 32 * 32;
    const int64_t begin = min(p.tokens, rank * per), end = min(p.tokens, begin + per);
    for (int pass = 0; pass < p.passes; ++pass) {
        sort_pass(p, sh, pass, per, begin, end, rank, ranks);
        __syncthreads();
    }
}

struct SumParams {
    const uint32_t* keys;
    const uint32_t* pos;
    uint32_t vocab;
    int chunk;                   // entries: 8, 16 or 32
    int64_t tokens, chunks;
    int dim, slices;             // slices of the columns, a warp's each
    int64_t ldo, ldt;
    float scale;
    int accumulate;
    int row_floats;              // of a partial sum: dim, rounded up to 4
    float* partial;              // [2][chunks][row_floats]: a chunk's part of a row that began
                                 // before it (0), and of one that goes on behind it (1)
    uint32_t* long_rows;         // their number, and from [1] on the chunks they begin in
};

// A row's columns c.. : scale * sum, or that added to what is there.  Into fp32 the memory
// system adds (each element once in a call, so no order matters), which no thread waits for.
template <typename G, int VEC>
__device__ __forceinline__ void write_columns(const SumParams& p, G* at, int64_t left, const float (&sum)[VEC]) {
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p.scale * sum[i];
    if (p.accumulate) {
        if constexpr (sizeof(G) == 4) {
            if (VEC >= 4 && left >= VEC) {
#pragma unroll
                for (int i = 0; i + 3 < VEC; i += 4)
                    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};"
                                 :: "l"(at + i), "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]) : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (i < left) asm volatile("red.global.add.f32 [%0], %1;" :: "l"(at + i), "f"(v[i]) : "memory");
            }
            return;
        } else {
            float old[VEC];
            load_values<G, VEC>(at, left, old);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] += old[i];
        }
    }
    store_values<G, VEC>(at, left, v);
}

// A warp per chunk and slice: 32 lanes x REP packs of VEC columns.  Bound by bytes, dout read
// once and the rows written: 16384 x 4096 bf16 35 us, 4 TB/s counted, eight rows in flight a
// warp.
template <typename T, typename G, int VEC, int REP>
__global__ void __launch_bounds__(kThreads)
embed_sum_kernel(const SumParams p, const T* __restrict__ dout, G* __restrict__ table) {
    constexpr int kAhead = 8;                    // rows in flight
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lane = threadIdx.x % 32, L = p.chunk;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    const int64_t chunk = unit / p.slices;
    const int slice = static_cast<int>(unit % p.slices);
    if (chunk >= p.chunks) return;
    const int64_t first = chunk * L;
    // the keys before, in and behind the chunk, and the positions of the latter
    const auto key_at = [&](int64_t e, bool want) { return want && e >= 0 && e < p.tokens ? p.keys[e] : p.vocab; };
    const uint32_t before = key_at(first - L + lane, lane < L);
    const uint32_t in = key_at(first + lane, lane < L);
    const uint32_t behind = key_at(first + L + lane, lane < L);
    const uint32_t pos_in = lane < L && first + lane < p.tokens ? p.pos[first + lane] : 0;
    const uint32_t pos_behind = lane < L && first + L + lane < p.tokens ? p.pos[first + L + lane] : 0;
    const unsigned all = 0xffffffffu, chunk_mask = L == 32 ? all : (1u << L) - 1u;
    const uint32_t key_first = __shfl_sync(all, in, 0), key_last = __shfl_sync(all, in, L - 1);
    const int valid = __popc(__ballot_sync(all, in < p.vocab));      // the others sort last
    if (valid == 0) return;
    // the first row: entries before the chunk and in it (no more than L each are looked at)
    const unsigned back_mask = __ballot_sync(all, lane < L && before == key_first);
    const unsigned run_mask = __ballot_sync(all, lane < L && in == key_first);
    const int back = L == 32 ? __clz(~back_mask) : __clz(~(back_mask << (32 - L)));
    const int run = run_mask == chunk_mask ? L : __ffs(~run_mask) - 1;
    const bool head_long = back > 0 && (back >= L || run == L || back + run > L);
    // the last one: its entries in the chunk and behind it
    const unsigned tail_mask = __ballot_sync(all, lane < L && in == key_last);
    const unsigned next_mask = __ballot_sync(all, lane < L && behind == key_last && key_last < p.vocab);
    const int tail = L == 32 ? __clz(~tail_mask) : __clz(~(tail_mask << (32 - L)));
    const int next = next_mask == chunk_mask ? L : __ffs(~next_mask) - 1;
    const bool is_head = run == L && back > 0;                       // the last row is the first, begun before
    const bool tail_long = !is_head && next > 0 && tail + next > L;
    const int begin = back > 0 && !head_long ? run : 0;              // (a short row begun before is done there)
    const int end = is_head || tail_long || valid < L ? valid : L + next;
    if (tail_long && slice == 0 && lane == 0) p.long_rows[1 + atomicAdd(p.long_rows, 1u)] = static_cast<uint32_t>(chunk);
    // the last entries of rows
    const uint32_t behind_first = __shfl_sync(all, behind, 0);
    const uint32_t in_next = __shfl_down_sync(all, in, 1), behind_next = __shfl_down_sync(all, behind, 1);
    const unsigned last_in = __ballot_sync(all, lane < L && in != (lane == L - 1 ? behind_first : in_next));
    const unsigned last_behind = __ballot_sync(all, lane == L - 1 || behind != behind_next);

    const int c0 = slice * 32 * VEC * REP + lane * VEC;              // pack k at c0 + k * 32 * VEC
    constexpr int kPairs = REP * VEC / 2;
    Pair sum[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) sum[j] = Pair(0.f, 0.f);
    for (int e0 = begin; e0 < end; e0 += kAhead) {
        Pack<T, VEC> row[kAhead][REP];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int e = e0 + u;
            const uint32_t at_in = __shfl_sync(all, pos_in, e & 31), at_behind = __shfl_sync(all, pos_behind, (e - L) & 31);
            const T* from = dout + (e < L ? at_in : at_behind) * p.ldo;
#pragma unroll
            for (int k = 0; k < REP; ++k) {
                const int c = c0 + k * 32 * VEC;
                if (e < end && c < p.dim) row[u][k] = load_pack<T, VEC>(from + c, p.dim - c);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int e = e0 + u;
            if (e >= end) break;
            Pair v[kPairs];
            to_pairs(row[u], v);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum[j] = add2(sum[j], v[j]);
            const bool last = e < L ? last_in >> e & 1u : last_behind >> (e - L) & 1u;
            if (!last && e != end - 1) continue;
            const bool to_head = e < run && head_long, to_tail = e == L - 1 && tail_long;
            const uint32_t key = __shfl_sync(all, e < L ? in : behind, (e < L ? e : e - L) & 31);
#pragma unroll
            for (int k = 0; k < REP; ++k) {
                const int c = c0 + k * 32 * VEC;
                float total[VEC];
                if constexpr (VEC == 1) {
                    float lo, hi;
                    sum[k / 2].get(lo, hi);
                    total[0] = k % 2 == 0 ? lo : hi;
                } else {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) sum[k * (VEC / 2) + j].get(total[2 * j], total[2 * j + 1]);
                }
                if (c < p.dim) {
                    if (to_head || to_tail)
                        store_values<float, VEC>(p.partial + ((to_head ? 0 : p.chunks) + chunk) * p.row_floats + c,
                                                 p.row_floats - c, total);
                    else
                        write_columns<G, VEC>(p, table + key * p.ldt + c, p.dim - c, total);
                }
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum[j] = Pair(0.f, 0.f);
        }
    }
}

// The rows with partial sums: a block takes one and 128 columns at a time, its warps the
// row's chunks in turn.
template <typename G, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const SumParams p, G* __restrict__ table) {
    constexpr int kWarps = kThreads / 32, kAhead = 4;
    __shared__ float4 part[kWarps][32];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int tiles = (p.dim + 127) / 128;
    const int64_t items = static_cast<int64_t>(*p.long_rows) * tiles;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t chunk = p.long_rows[1 + item / tiles];
        const int c = static_cast<int>(item % tiles) * 128 + lane * 4;
        const uint32_t key = p.keys[(chunk + 1) * p.chunk - 1];
        // the chunks behind that begin with the row
        int64_t more = 0;
        for (;;) {
            const int64_t k = chunk + 1 + more + lane;
            const unsigned same = __ballot_sync(0xffffffffu, k < p.chunks && p.keys[k * p.chunk] == key);
            more += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
            if (same != 0xffffffffu) break;
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < p.dim) {
            // part 0 is the first chunk's, part j > 0 that of the j-th chunk behind it
            for (int64_t j = warp; j <= more; j += kAhead * kWarps) {
                float4 v[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t k = j + u * kWarps;
                    v[u] = k <= more ? *reinterpret_cast<const float4*>(
                                           p.partial + ((k == 0 ? p.chunks : 0) + chunk + k) * p.row_floats + c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    sum.x += v[u].x;
                    sum.y += v[u].y;
                    sum.z += v[u].z;
                    sum.w += v[u].w;
                }
            }
        }
        part[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && c < p.dim) {
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = part[w][lane];
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            G* at = table + key * p.ldt + c;
            if constexpr (ALIGNED) {
                const float v[4] = {sum.x, sum.y, sum.z, sum.w};
                write_columns<G, 4>(p, at, p.dim - c, v);
            } else {
                const float v[4] = {sum.x, sum.y, sum.z, sum.w};
                for (int i = 0; i < 4; ++i) {
                    const float one[1] = {v[i]};
                    write_columns<G, 1>(p, at + i, p.dim - c - i, one);
                }
            }
        }
        __syncthreads();
    }
}

// Entries a chunk: the largest of 32, 16 and 8 that leaves four warps or more to each of an
// SM's four schedulers.
int chunk_of(int64_t tokens, int slices, int sms) {
    int chunk = 32;
    while (chunk > 8 && (tokens / chunk) * slices < int64_t{16} * sms) chunk /= 2;
    return chunk;
}

// The most chunks of any call of up to `tokens` tokens.
int64_t most_chunks(int64_t tokens, int slices, int sms) {
    int64_t most = 0;
    for (int64_t t = tokens;;) {
        const int chunk = chunk_of(t, slices, sms);
        const int64_t n = (t + chunk - 1) / chunk;
        if (n > most) most = n;
        if (chunk == 8) return most;
        // fewer tokens: the next smaller chunk begins below the limit of this one
        t = (int64_t{16} * sms + slices - 1) / slices * chunk - 1;
    }
}

// Columns of a warp's slice.
int slice_columns(int elem, bool aligned) { return aligned ? 32 * 16 / elem : 32 * 4; }

template <typename T, typename G, int VEC, int REP>
gemm_status_t sum_rows(SumParams s, int sms, const T* dout, G* table, Queue queue) {
    const int64_t units = s.chunks * s.slices, warps = kThreads / 32;
    const gemm_status_t st =
        launch<embed_sum_kernel<T, G, VEC, REP>>((units + warps - 1) / warps, kThreads, 0, queue, 1, s, dout, table);
    if (st != GEMM_OK || s.tokens <= s.chunk) return st;     // (no row is longer than a chunk)
    return launch<embed_join_kernel<G, (VEC > 1)>>(4 * sms, kThreads, 0, queue, 1, s, table);
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
    if (vocab < 1 || vocab > INT32_MAX || dim < 1 || dim > gbt::kMostColumns ||
        max_tokens < 0 || max_tokens > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    int device = 0, sms = 0;
    gemm_status_t st = gbt::begin_plan(&device, &sms);
    if (st != GEMM_OK) return st;
    const auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
    const size_t list = padded(static_cast<size_t>(max_tokens) * 4);
    int64_t chunks = 0;
    for (int aligned = 0; aligned < 2; ++aligned) {
        const int columns = gbt::slice_columns(gbt::elem_bytes(elem), aligned != 0);
        const int64_t n = gbt::most_chunks(max_tokens, static_cast<int>((dim + columns - 1) / columns), sms);
        if (n > chunks) chunks = n;
    }
    const size_t rows = padded(static_cast<size_t>(chunks + 1) * 4);
    const size_t sums = static_cast<size_t>(chunks) * 2 * static_cast<size_t>((dim + 3) / 4 * 4) * 4;
    void* memory = nullptr;
    st = gbt::allocate(&memory, 256 + 4 * list + rows + sums);
    if (st != GEMM_OK) return st;
    if (cudaFuncSetAttribute(gbt::embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sizeof(gbt::SortShared)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(memory);
        return GEMM_ERR_LAUNCH;
    }
    gemm_embed_plan* p = new (std::nothrow) gemm_embed_plan();
    if (!p || gbt::clear_now(memory, 256) != GEMM_OK) {
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
    p->long_rows = reinterpret_cast<uint32_t*>(at);
    p->partial = reinterpret_cast<float*>(at + rows);
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
    const gbt::Queue queue{stream, p->device};
    const gbt::LookupParams q{ids,  static_cast<int>(id_type), padding, tokens, p->vocab, ldt, ldo, scale,
                              static_cast<int>(p->dim), 0, p->error_word};
    const bool vec = gbt::rows_aligned(table, ldt, e) && gbt::rows_aligned(out, ldo, e);
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        const T* from = static_cast<const T*>(table);
        T* to = static_cast<T*>(out);
        return vec ? gbt::lookup<T, kVec>(q, p->num_sms, from, to, queue)
                   : gbt::lookup<T, 1>(q, p->num_sms, from, to, queue);
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
    const gbt::Queue queue{stream, p->device};
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
    q.long_rows = p->long_rows;
    q.fill_shift = -1;
    q.table = dtable;
    q.row_bytes = p->dim * g;
    q.stride_bytes = ldt * g;
    q.vector_rows = gbt::rows_aligned(dtable, ldt, g);
    // the sorting cluster: up to kSortBlock tokens a block
    int ranks = 1;
    while (ranks < gbt::kMaxCluster && ranks * gbt::kSortBlock < tokens) ranks *= 2;
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
    st = gbt::launch<gbt::embed_sort_kernel>(grid, gbt::kSortThreads, sizeof(gbt::SortShared), queue, ranks, q,
                     ranks);
    if (st != GEMM_OK || tokens == 0) return st;

    gbt::SumParams s = {};
    s.keys = p->keys[0];
    s.pos = p->pos[0];
    s.vocab = q.vocab;
    const int e = gbt::elem_bytes(p->elem);
    const bool vec = gbt::rows_aligned(dout, ldo, e) && q.vector_rows;
    const int columns = gbt::slice_columns(e, vec);
    s.tokens = tokens;
    s.dim = static_cast<int>(p->dim);
    s.slices = static_cast<int>((p->dim + columns - 1) / columns);
    s.chunk = gbt::chunk_of(tokens, s.slices, p->num_sms);
    s.chunks = (tokens + s.chunk - 1) / s.chunk;
    s.ldo = ldo;
    s.ldt = ldt;
    s.scale = scale;
    s.accumulate = accumulate;
    s.row_floats = static_cast<int>((p->dim + 3) / 4 * 4);
    s.partial = p->partial;
    s.long_rows = p->long_rows;
    return gbt::with_elem(p->elem, [&](auto t) {
        using T = decltype(t);
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        const auto run = [&](auto v) {
            using G = decltype(v);
            const T* d = static_cast<const T*>(dout);
            G* w = static_cast<G*>(dtable);
            return vec ? gbt::sum_rows<T, G, kVec, 1>(s, p->num_sms, d, w, queue)
                       : gbt::sum_rows<T, G, 1, 4>(s, p->num_sms, d, w, queue);
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
