// ffn_gated.cu -- the gated product H = act(X Wg^T) * (X Wu^T) of gemm_ffn.h, and its gradients.
#include <new>
#include <type_traits>

#include "ffn_mma.cuh"
#include "gemm_launch.h"

struct gemm_gated_plan {
    int64_t M, F, K;
    gemm_elem_t elem;
    gemm_activation_t act;
    gbf::PlanBase base;
    gbf::FewChoice choice;       // of the forward kernel
    int width;                   // of the tiles of the kernel of many rows
    gemm_plan_t dx, dw;          // the gradients' products
};

namespace gbf {
namespace {

constexpr int kPairStages = 6;
constexpr int kTileF = 128;                       // columns of H in a tile, at most
constexpr int kPairEpilogue = 8;                  // epilogue warps: two to each quarter of the TMEM lanes
constexpr int kPairThreads = 64 + 32 * kPairEpilogue;
using PairLayout = SmemLayout2<2 * kTileF, kPairStages, 1>;
static_assert(kPairEpilogue * PairLayout::kStoreBufBytes <= PairLayout::kStagingBytes, "a store buffer a warp");

struct GatedParams {
    int32_t M, F;
    int32_t width;               // columns of H in a tile: 64 to 128, a multiple of 16
    int32_t num_kb, m_blocks, num_units;
    uint32_t idesc, tx_extra;
    int32_t act;
    void* H;
    void* gate_up;               // NULL: not kept
    int32_t* error_word;
    uint64_t timeout_ns;
    RasterDiv rd;
};

// Many rows: a pair of SMs computes 256 rows of X times 128 rows of each half of W as one
// tcgen05.mma of 256 x 256.  In such a pair each CTA brings half of the B operand, so the
// leader brings the gate's rows and its peer the other half's: both products of one column of
// H end in the same TMEM lane, columns c and 128 + c, and the epilogue has them side by side.
// The main loop is the plain product's (gemm_kernel_2cta.cuh), bound by the tensor cores; eight
// epilogue warps of 64 columns keep the activation behind it.  Narrower tiles (a smaller N) take the place
// of a last wave that would be nearly empty; their last columns, less than 64, are stored by
// each thread from its row.
template <int OUT>
__global__ void __launch_bounds__(kPairThreads, 1)
    gated_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_gate,
                      const __grid_constant__ CUtensorMap tmap_up, const __grid_constant__ CUtensorMap tmap_h,
                      const __grid_constant__ CUtensorMap tmap_keep_gate, const __grid_constant__ CUtensorMap tmap_keep_up,
                      const GatedParams p) {
    using L = PairLayout;
    constexpr int kStages = kPairStages;
    constexpr int kBN = 2 * kTileF;
    constexpr uint32_t kTmemCols = 2 * kBN;
    const uint32_t pair_tx = 2 * (L::kASlotBytes + static_cast<uint32_t>(p.width) * kRowBytes);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem), ring_b = ring + kStages * L::kASlotBytes;
    const uint32_t staging = ring + L::kRingBytes;
    SharedCtl<kStages>* ctl = reinterpret_cast<SharedCtl<kStages>*>(smem + L::kRingBytes + L::kStagingBytes);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int32_t pair = static_cast<int32_t>(blockIdx.x >> 1), npairs = static_cast<int32_t>(gridDim.x >> 1);

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_gate);
        prefetch_tmap(&tmap_up);
        prefetch_tmap(&tmap_h);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&ctl->tmem_full[b]), 1);
            mbar_init(smem_addr(&ctl->tmem_empty[b]), 2 * kPairEpilogue);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Watch watch{&ctl->abort, p.error_word, p.timeout_ns};
    if (!leader && threadIdx.x == 0) {
        // the leader's MMAs address the peer's TMEM with the leader's address
        if (ld_dsmem_u32(map_to_rank(smem_addr(&ctl->tmem_base), 0)) != tmem_base) {
            atomicCAS(p.error_word, 0, kSitePairTmem);
            ctl->abort = 1;
        }
    }
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == 0) {
        if (elect_one_sync()) {
            const CUtensorMap* tmap_w = leader ? &tmap_gate : &tmap_up;
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int32_t u = pair; ok && u < p.num_units; u += npairs) {
                int32_t m_blk, f_blk;
                raster_tile_fast(p.m_blocks, p.rd, u, &m_blk, &f_blk);
                const int32_t x_row = (2 * m_blk + static_cast<int32_t>(rank)) * kBM, w_row = f_blk * p.width;
                for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (issued >= kStages &&
                        !wait_phase(smem_addr(&ctl->empty[stage]), phase ^ 1u, watch, kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = smem_addr(&ctl->full[stage]);
                    if (leader) mbar_arrive_expect_tx(full, pair_tx + p.tx_extra);
                    const uint32_t full_lead = map_to_rank(full, 0);
                    tma_load_2d_pair(ring + stage * L::kASlotBytes, &tmap_x, full_lead, kb * kBK, x_row);
                    tma_load_2d_pair(ring_b + stage * L::kBTileBytes, tmap_w, full_lead, kb * kBK, w_row);
                    issued = issued < kStages ? issued + 1 : kStages;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // both CTAs' copies count on the leader's barriers: they land before the pair can leave
            for (int i = 0; i < issued; ++i) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    phase ^= 1u;
                }
                if (leader) wait_phase_unwind(smem_addr(&ctl->full[stage]), phase, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && elect_one_sync()) {
            int stage = 0;
            uint32_t phase = 0, turn = 0;
            bool ok = true;
            for (int32_t u = pair; ok && u < p.num_units; u += npairs, ++turn) {
                const uint32_t buf = turn & 1u;
                if (turn >= 2 && !wait_phase_cluster(smem_addr(&ctl->tmem_empty[buf]), ((turn >> 1) & 1u) ^ 1u, watch,
                                                     kSiteMmaTmemEmpty))
                    break;
                tc_fence_after();
                for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_phase(smem_addr(&ctl->full[stage]), phase, watch, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = sw128_kmajor_desc(ring + stage * L::kASlotBytes);
                    const uint64_t b_desc = sw128_kmajor_desc(ring_b + stage * L::kBTileBytes);
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        umma_f16_pair(tmem_base + buf * kBN, a_desc + 2 * k, b_desc + 2 * k, p.idesc,
                                      kb > 0 || k > 0 ? 1u : 0u);
                    umma_commit_pair(smem_addr(&ctl->empty[stage]), 3);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (ok) umma_commit_pair(smem_addr(&ctl->tmem_full[buf]), 3);
            }
            umma_commit_pair(smem_addr(&ctl->drain), 1);
            wait_phase_unwind(smem_addr(&ctl->drain), 0, 100000000ull);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, c = ((warp - 2) >> 2) * 64;
        const uint32_t lanes_at = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c);
        const uint32_t store_buf = staging + static_cast<uint32_t>((warp - 2) * L::kStoreBufBytes);
        uint32_t turn = 0;
        const int cols = min(64, p.width - c);           // of the warp
        // its columns of 32 rows, 32 at a time: 64 through the warp's buffer, fewer from the registers
        // to row y + lane of a matrix whose rows are ld apart
        const auto store = [&](const CUtensorMap* map, void* to, int64_t ld, int32_t x, int32_t y, auto columns) {
            const bool whole = cols == 64;
            if (whole) {
                if (lane == 0) bulk_wait_group_read<0>();
                __syncwarp();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h * 32 >= cols) break;
                uint32_t v[32], w[16];
                columns(h * 32, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack2<OUT>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                if (whole) {
                    stage_store_row(store_buf, lane, h * 4, w, 4);
                } else if (y + lane < p.M) {
                    uint16_t* row = static_cast<uint16_t*>(to) + static_cast<int64_t>(y + lane) * ld + x + h * 32;
#pragma unroll
                    for (int g = 0; g < 4; ++g)              // (F % 8 == 0)
                        if (h * 32 + g * 8 < cols && x + h * 32 + g * 8 < p.F)
                            *reinterpret_cast<uint4*>(row + g * 8) = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
                }
            }
            if (!whole) return;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, store_buf, x, y);
                bulk_commit_group();
            }
        };
        for (int32_t u = pair; u < p.num_units; u += npairs, ++turn) {
            int32_t m_blk, f_blk;
            raster_tile_fast(p.m_blocks, p.rd, u, &m_blk, &f_blk);
            const int32_t y = (2 * m_blk + static_cast<int32_t>(rank)) * kBM + quad * 32, x = f_blk * p.width + c;
            const uint32_t buf = turn & 1u, gate_at = lanes_at + buf * kBN, up_at = gate_at + static_cast<uint32_t>(p.width);
            if (!wait_phase(smem_addr(&ctl->tmem_full[buf]), (turn >> 1) & 1u, watch, kSiteEpiTmemFull)) break;
            tc_fence_after();
            if (y < p.M && x < p.F && cols > 0) {        // (the whole warp)
                const auto products = [&](uint32_t at) {
                    return [=](int col, uint32_t (&v)[32]) {
                        tmem_ld_32x32b_x32(at + static_cast<uint32_t>(col), v);
                        tmem_ld_wait();
                    };
                };
                if (p.gate_up) {
                    store(&tmap_keep_gate, p.gate_up, 2 * static_cast<int64_t>(p.F), x, y, products(gate_at));
                    store(&tmap_keep_up, static_cast<uint16_t*>(p.gate_up) + p.F, 2 * static_cast<int64_t>(p.F), x, y,
                          products(up_at));
                }
                with_act(p.act, [&](auto act) {
                    store(&tmap_h, p.H, p.F, x, y, [&](int col, uint32_t (&v)[32]) {
                        uint32_t g[32];
                        tmem_ld_32x32b_x32(gate_at + static_cast<uint32_t>(col), g);
                        tmem_ld_32x32b_x32(up_at + static_cast<uint32_t>(col), v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint(gate_fn<decltype(act)::value>(__uint_as_float(g[i])) * __uint_as_float(v[i]));
                    });
                });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(smem_addr(&ctl->tmem_empty[buf]));
        }
    }

    tc_fence_before();
    cluster_sync_all();                              // the pair's MMAs, TMEM reads and copies are all finished
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    } else if (warp >= 2) {
        if (lane == 0) bulk_wait_group_read<0>();    // the stores have read their buffers
        __syncwarp();
    }
}

// ---------------------------------------------------------------- gradients of the gate

constexpr int kGradThreads = 256;

// (act(g), act'(g))
template <int ACT>
__device__ __forceinline__ float2 gate_and_slope(float g) {
    if constexpr (ACT == GEMM_ACT_RELU) return make_float2(gate_fn<ACT>(g), g > 0.f ? 1.f : 0.f);
    if constexpr (ACT == GEMM_ACT_GELU) {
        const float e = bell(g), phi = normal_cdf(g, e);
        return make_float2(g * phi, e == 0.f ? phi : fmaf(g, 0.39894228f * e, phi));   // (inf * 0)
    }
    if constexpr (ACT == GEMM_ACT_SILU) {
        const float s = sigmoid(g), rest = sigmoid(-g);
        return make_float2(g * s, rest == 0.f ? s : s * fmaf(g, rest, 1.f));
    }
    return make_float2(g, 1.f);
}

// dgate_up from gate_up and dH, eight columns a thread; bound by memory.
template <typename T, int ACT>
__global__ void __launch_bounds__(kGradThreads) gate_grad_kernel(const T* gate_up, const T* dh, T* dgate_up, int64_t F,
                                                                int chunks) {
    const int64_t row = blockIdx.x / static_cast<unsigned>(chunks);
    const int64_t c = (static_cast<int64_t>(blockIdx.x % static_cast<unsigned>(chunks)) * kGradThreads + threadIdx.x) * 8;
    gbt::wait_for_previous_kernel();
    gbt::let_next_kernel_start();
    if (c >= F) return;
    gbt::Eight<T> g, u, d;
    g.template load<true>(gate_up + row * 2 * F + c, 8);
    u.template load<true>(gate_up + row * 2 * F + F + c, 8);
    d.template load<true>(dh + row * F + c, 8);
    gbt::Pair gate[4], up[4], grad[4];
    g.get(gate);
    u.get(up);
    d.get(grad);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        gate[i].get(lo, hi);
        const float2 a = gate_and_slope<ACT>(lo), b = gate_and_slope<ACT>(hi);
        gate[i] = gbt::mul2(gbt::mul2(grad[i], up[i]), gbt::Pair(a.y, b.y));
        up[i] = gbt::mul2(grad[i], gbt::Pair(a.x, b.x));
    }
    g.set(gate);
    u.set(up);
    g.template store<true>(dgate_up + row * 2 * F + c, 8);
    u.template store<true>(dgate_up + row * 2 * F + F + c, 8);
}

template <typename T>
gemm_status_t gate_grad(const gemm_gated_plan* p, const void* gate_up, const void* dh, void* dgate_up, gbt::Queue queue) {
    const int chunks = static_cast<int>((p->F / 8 + kGradThreads - 1) / kGradThreads);
    const auto go = [&](auto act) {
        return gbt::launch<gate_grad_kernel<T, decltype(act)::value>>(p->M * chunks, kGradThreads, 0, queue, 1,
                                                                      static_cast<const T*>(gate_up), static_cast<const T*>(dh),
                                                                      static_cast<T*>(dgate_up), p->F, chunks);
    };
    switch (p->act) {
        case GEMM_ACT_RELU: return go(std::integral_constant<int, GEMM_ACT_RELU>());
        case GEMM_ACT_GELU: return go(std::integral_constant<int, GEMM_ACT_GELU>());
        case GEMM_ACT_SILU: return go(std::integral_constant<int, GEMM_ACT_SILU>());
        default: return go(std::integral_constant<int, GEMM_ACT_NONE>());
    }
}

// ---------------------------------------------------------------- launches

template <int OUT>
bool prepare() {
    return allow_shared<gated_pair_kernel<OUT>>(PairLayout::kTotal) &&
           allow_shared<few_rows_kernel<false, OUT, 32>>(FewLayout<32>::kTotal) &&
           allow_shared<few_rows_kernel<false, OUT, 128>>(FewLayout<128>::kTotal);
}

template <int OUT>
gemm_status_t forward_few(const gemm_gated_plan* p, const void* X, const void* W, void* H, void* gate_up, gbt::Queue queue) {
    const auto type = OUT == kOutF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int box = p->M <= 32 ? 32 : kTileSide;
    CUtensorMap x, gate, up;
    if (!encode_map(&x, type, 2, X, p->M, p->K, p->K, box) ||
        !encode_map(&gate, type, 2, W, p->F, p->K, p->K, kTileSide / 2) ||
        !encode_map(&up, type, 2, static_cast<const uint16_t*>(W) + p->F * p->K, p->F, p->K, p->K, kTileSide / 2))
        return GEMM_ERR_TENSORMAP;
    FewParams f{};
    f.M = static_cast<int32_t>(p->M);
    f.N = static_cast<int32_t>(p->F);
    f.num_kb = static_cast<int32_t>((p->K + kBK - 1) / kBK);
    f.m_blocks = static_cast<int32_t>((p->M + kTileSide - 1) / kTileSide);
    const int64_t tiles = f.m_blocks * ((p->F + kTileSide / 2 - 1) / (kTileSide / 2));
    f.slices = p->choice.slices;
    f.kb_per_slice = p->choice.kb_per_slice;
    f.idesc = descriptor(OUT == kOutF16 ? 0 : 1, kTileSide, kTileSide);
    f.tx_extra = p->base.tx_extra;
    f.act = p->act;
    f.out = H;
    f.gate_up = gate_up;
    f.error_word = p->base.error_word;
    f.timeout_ns = p->base.timeout_ns;
    if (box == 32)
        return gbt::launch<few_rows_kernel<false, OUT, 32>>(tiles * f.slices, kThreads, FewLayout<32>::kTotal, queue, f.slices, x,
                                                            gate, up, f);
    return gbt::launch<few_rows_kernel<false, OUT, 128>>(tiles * f.slices, kThreads, FewLayout<128>::kTotal, queue, f.slices, x,
                                                         gate, up, f);
}

template <int OUT>
gemm_status_t forward_many(const gemm_gated_plan* p, const void* X, const void* W, void* H, void* gate_up, gbt::Queue queue) {
    const auto type = OUT == kOutF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t M = p->M, F = p->F, K = p->K;
    CUtensorMap x, gate, up, h, keep_gate, keep_up;
    uint16_t* keep = static_cast<uint16_t*>(gate_up ? gate_up : H);
    const int64_t stride = gate_up ? 2 * F : F, second = gate_up ? F : 0;
    if (!encode_map(&x, type, 2, X, M, K, K, kTileSide) || !encode_map(&gate, type, 2, W, F, K, K, p->width) ||
        !encode_map(&up, type, 2, static_cast<const uint16_t*>(W) + F * K, F, K, K, p->width) ||
        !encode_map(&h, type, 2, H, M, F, F, 32) || !encode_map(&keep_gate, type, 2, keep, M, F, stride, 32) ||
        !encode_map(&keep_up, type, 2, keep + second, M, F, stride, 32))
        return GEMM_ERR_TENSORMAP;
    GatedParams g{};
    g.M = static_cast<int32_t>(M);
    g.F = static_cast<int32_t>(F);
    g.width = p->width;
    g.num_kb = static_cast<int32_t>((K + kBK - 1) / kBK);
    g.m_blocks = static_cast<int32_t>((M + 2 * kBM - 1) / (2 * kBM));
    const int32_t f_blocks = static_cast<int32_t>((F + p->width - 1) / p->width);
    g.num_units = g.m_blocks * f_blocks;
    g.idesc = descriptor(OUT == kOutF16 ? 0 : 1, 2 * kBM, 2 * p->width);
    g.tx_extra = p->base.tx_extra;
    g.act = p->act;
    g.H = H;
    g.gate_up = gate_up;
    g.error_word = p->base.error_word;
    g.timeout_ns = p->base.timeout_ns;
    // bands of eight row blocks: the 76 pairs cover about 8 x 9 tiles at a time
    g.rd = make_raster_div(g.m_blocks, f_blocks, g.m_blocks < 8 ? g.m_blocks : 8);
    const int pairs = p->base.num_sms / 2;
    return gbt::launch<gated_pair_kernel<OUT>>(2 * (g.num_units < pairs ? g.num_units : pairs), kPairThreads, PairLayout::kTotal,
                                               queue, 2, x, gate, up, h, keep_gate, keep_up, g);
}

template <int OUT>
gemm_status_t forward(const gemm_gated_plan* p, const void* X, const void* W, void* H, void* gate_up, gbt::Queue queue) {
    return p->choice.slices > 0 ? forward_few<OUT>(p, X, W, H, gate_up, queue)
                                : forward_many<OUT>(p, X, W, H, gate_up, queue);
}

// The width of the tiles of the kernel of many rows, 64 to 128 columns of H: the one whose waves over the SM
// pairs take the least, where a tile of width w takes 0.35 + 0.65 w / 128 of a full one (1000 x 3000 x 1000 17.8 us
// with 128, 15.0 with 80; 1024 x 4096 x 2048 22.7 with 128, 21.1 with 112; from some waves on 128 is best:
// 4096 x 8192 x 4096 277 against 286; inputs in L2 where they fit).  *waves: what they take, in waves of full tiles.
int tile_width(int64_t M, int64_t F, int num_sms, double* waves) {
    const int64_t pairs = num_sms / 2, rows = (M + 2 * kBM - 1) / (2 * kBM);
    int best = kTileF;
    for (int w = kTileF; w >= 64; w -= 16) {
        const int64_t tiles = rows * ((F + w - 1) / w);
        const double time = static_cast<double>((tiles + pairs - 1) / pairs) * (0.35 + 0.65 * w / kTileF);
        if (w == kTileF || time < 0.97 * *waves) {
            best = w;
            *waves = time;
        }
    }
    return best;
}

FewChoice choose(int64_t M, int64_t F, int64_t K, double pair_waves, int num_sms) {
    constexpr FewRates kRates{0.22, 0.35, 1.35, 0.29, 1.0};
    const int64_t few = ((M + kTileSide - 1) / kTileSide) * ((F + kTileSide / 2 - 1) / (kTileSide / 2));
    return choose_kernel(M, few, pair_waves, static_cast<int>((K + kBK - 1) / kBK), 4.0 * F * K, num_sms, kRates);
}

bool misaligned(const void* a, const void* b, const void* c, const void* d) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
             reinterpret_cast<uintptr_t>(d)) & 15u) != 0;
}

}  // namespace
}  // namespace gbf

extern "C" {

gemm_status_t gemm_gated_plan_create(int64_t M, int64_t F, int64_t K, gemm_elem_t elem, gemm_activation_t act,
                                     gemm_gated_plan_t* plan) {
    using namespace gbf;
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if ((elem != GEMM_ELEM_F16 && elem != GEMM_ELEM_BF16) || act < GEMM_ACT_NONE || act > GEMM_ACT_SILU)
        return GEMM_ERR_UNSUPPORTED;
    if (M < 0 || F < 0 || K < 0 || M > INT32_MAX || F > INT32_MAX / 2 || K > INT32_MAX) return GEMM_ERR_INVALID_ARG;
    if (F % 8 != 0 || K % 8 != 0) return GEMM_ERR_ALIGNMENT;
    // (tiles of the products, and blocks of the gate's gradients, in 32 bits)
    if ((M / 128 + 1) * (F / 64 + 1) > (int64_t{1} << 27) || M * (F / (8 * kGradThreads) + 1) > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    gemm_gated_plan* p = new (std::nothrow) gemm_gated_plan();
    if (!p) return GEMM_ERR_OOM;
    p->M = M;
    p->F = F;
    p->K = K;
    p->elem = elem;
    p->act = act;
    gemm_status_t st = open_plan(&p->base);
    if (st != GEMM_OK) {
        delete p;
        return st;
    }
    double waves = 0;
    p->width = tile_width(M, F, p->base.num_sms, &waves);
    p->choice = choose(M, F, K, waves, p->base.num_sms);
    const gemm_dtype_t type = elem == GEMM_ELEM_F16 ? GEMM_F16 : GEMM_BF16;
    if (!(elem == GEMM_ELEM_F16 ? prepare<kOutF16>() : prepare<kOutBF16>())) st = GEMM_ERR_LAUNCH;
    if (st == GEMM_OK) st = gemm_plan_create(M, K, 2 * F, type, GEMM_LAYOUT_NN, &p->dx);
    if (st == GEMM_OK) st = gemm_plan_create(2 * F, K, M, type, GEMM_LAYOUT_NT, &p->dw);
    if (st != GEMM_OK) {
        gemm_gated_plan_destroy(p);
        return st;
    }
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_gated_forward(gemm_gated_plan_t p, const void* X, const void* W, void* H, void* gate_up, void* stream) {
    using namespace gbf;
    if (!p) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = gbt::check_device(p->base.device);
    if (st != GEMM_OK) return st;
    if (p->M == 0 || p->F == 0) return GEMM_OK;
    if (!H || (p->K > 0 && (!X || !W))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, W, H, gate_up)) return GEMM_ERR_ALIGNMENT;
    if (p->K == 0) {
        if (launch_zero_fill(H, p->M * p->F * 2, p->base.num_sms, static_cast<cudaStream_t>(stream)) != cudaSuccess ||
            (gate_up && launch_zero_fill(gate_up, p->M * p->F * 4, p->base.num_sms, static_cast<cudaStream_t>(stream)) != cudaSuccess)) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        return GEMM_OK;
    }
    const gbt::Queue queue{stream, p->base.device};
    return p->elem == GEMM_ELEM_F16 ? forward<kOutF16>(p, X, W, H, gate_up, queue)
                                    : forward<kOutBF16>(p, X, W, H, gate_up, queue);
}

gemm_status_t gemm_gated_backward(gemm_gated_plan_t p, const void* X, const void* W, const void* gate_up, const void* dH,
                                  void* dgate_up, void* dX, void* dW, void* stream) {
    using namespace gbf;
    if (!p) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = gbt::check_device(p->base.device);
    if (st != GEMM_OK) return st;
    const bool some = p->M > 0 && p->F > 0;
    if (some && (!gate_up || !dH || !dgate_up)) return GEMM_ERR_INVALID_ARG;
    if ((dX && some && p->K > 0 && !W) || (dW && some && p->K > 0 && !X)) return GEMM_ERR_INVALID_ARG;
    if (misaligned(X, W, gate_up, dH) || misaligned(dgate_up, dX, dW, nullptr)) return GEMM_ERR_ALIGNMENT;
    const gbt::Queue queue{stream, p->base.device};
    // (dgate_up is rounded to the type before its two products, whose operands have 16 bits: in bf16 at 4096 x 8192 x
    // 4096 dX and dW are 2.4e-3 from 64 bits in the norm, 1.7e-3 with 32-bit operands, which would halve the rate or more)
    if (some)
        st = p->elem == GEMM_ELEM_F16 ? gate_grad<__half>(p, gate_up, dH, dgate_up, queue)
                                      : gate_grad<__nv_bfloat16>(p, gate_up, dH, dgate_up, queue);
    if (st == GEMM_OK && dX) st = gemm_run(p->dx, dgate_up, W, dX, stream);
    if (st == GEMM_OK && dW) st = gemm_run(p->dw, dgate_up, X, dW, stream);
    return st;
}

gemm_status_t gemm_gated_plan_set_timeout(gemm_gated_plan_t p, uint64_t ns) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    p->base.timeout_ns = ns ? ns : gbf::kWaitLimitNs;
    gemm_plan_set_timeout(p->dx, ns);
    return gemm_plan_set_timeout(p->dw, ns);
}

gemm_status_t gemm_gated_plan_set_wait_test(gemm_gated_plan_t p, uint32_t extra_bytes) {
    if (!p || extra_bytes > 4096 || (extra_bytes & 15u)) return GEMM_ERR_INVALID_ARG;
    p->base.tx_extra = extra_bytes;
    gemm_plan_set_wait_test(p->dx, extra_bytes);
    return gemm_plan_set_wait_test(p->dw, extra_bytes);
}

gemm_status_t gemm_gated_plan_check(gemm_gated_plan_t p, void* stream) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = gbf::check_plan(&p->base, stream);
    for (gemm_plan_t g : {p->dx, p->dw}) {           // (each reads and clears its own word)
        const gemm_status_t s = gemm_plan_check(g, stream);
        if (st == GEMM_OK) st = s;
    }
    return st;
}

gemm_status_t gemm_gated_plan_destroy(gemm_gated_plan_t p) {
    if (!p) return GEMM_OK;
    gemm_status_t st = gbf::close_plan(&p->base);
    for (gemm_plan_t g : {p->dx, p->dw}) {
        const gemm_status_t s = gemm_plan_destroy(g);
        if (st == GEMM_OK) st = s;
    }
    delete p;
    return st;
}

}  // extern "C"
