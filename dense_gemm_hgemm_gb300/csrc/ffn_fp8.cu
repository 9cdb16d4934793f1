// ffn_fp8.cu -- the product of e4m3 matrices with a scale for each 128 elements (gemm_ffn.h).
#include <new>
#include <type_traits>

#include "ffn_mma.cuh"
#include "gemm_launch.h"

struct gemm_fp8_plan {
    int64_t M, N, K;
    gemm_elem_t out;
    gemm_scale_t b_scales;
    gbf::PlanBase base;
    gbf::FewChoice choice;       // of the kernel (by squares)
    int width;                   // of the tiles of the kernel of many rows
};

namespace gbf {
namespace {

constexpr int kSumWarps = 8;                      // of a CTA
constexpr int kFirstSumWarp = 4;                  // after the copies', the MMAs' and the column scales' two
constexpr int kPairThreads = 32 * (kFirstSumWarp + kSumWarps);
// Registers of a thread: 168 at the launch; the first warpgroup's go to the other two.
constexpr int kLaunchRegisters = 168, kFewRegisters = 72, kSumRegisters = 216;
static_assert(128 * kFewRegisters + 256 * kSumRegisters <= kPairThreads * kLaunchRegisters, "registers of the block");

// Tiles of 256 rows by BN columns (BYROW: B's scales go by rows).
template <bool BYROW, int BN>
struct Fp8Layout {
    static constexpr int kBN = BN;
    static constexpr int kTurns = 512 / kBN;                           // accumulators: all of TMEM
    static constexpr int kStages = BN == 128 && !BYROW ? 7 : 5;
    static constexpr int kBSlot = kBN / 2 * kRowBytes;                 // this CTA's half of B's rows
    static constexpr int kRing = kStages * (kTileSlot + kBSlot);
    static constexpr int kStoreBuf = 32 * kRowBytes;
    static constexpr int kStoreBufs = BN / 128;                        // of a warp: one for 64 columns
    static constexpr int kStaging = kSumWarps * kStoreBufs * kStoreBuf;
    static constexpr int kScaleSlot = 2 * kTileSide * 16;              // BYROW: of 128 columns and 128 rows, four steps
    static constexpr int kTotal = 1024 + kRing + kStaging + 256 + (BYROW ? 4 * kScaleSlot : 0);
    static_assert(kTotal <= 232448, "exceeds the 227 KiB a CTA may use");
};

struct Fp8Params {
    int32_t M, N;
    int32_t num_kb, m_blocks, num_units;
    uint32_t idesc, tx_extra;
    bool whole_scales;                            // by rows: their rows move in fours
    const float* a_scales;
    const float* b_scales;
    int32_t* error_word;
    uint64_t timeout_ns;
    RasterDiv rd;
};

// One scale on its way to shared memory; and this thread's arrival on a barrier once all that it
// has asked for so far is there.
__device__ __forceinline__ void fetch_scale(uint32_t to, const float* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void fetch_scales(uint32_t to, const float* from) {      // four, 16-byte aligned
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void arrive_when_fetched(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ gbt::Pair ld_shared_twice(uint32_t saddr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(saddr) : "memory");
    return gbt::Pair(v, v);
}
// Values 16 bytes apart.
__device__ __forceinline__ gbt::Pair ld_shared_pair(uint32_t saddr) {
    float lo, hi;
    asm volatile("ld.shared.f32 %0, [%2];\n\tld.shared.f32 %1, [%2 + 16];" : "=f"(lo), "=f"(hi) : "r"(saddr) : "memory");
    return gbt::Pair(lo, hi);
}
__device__ __forceinline__ void st_shared_u1(uint32_t saddr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

template <int STAGES>
struct Fp8Ctl {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t sums_full[4], sums_empty[4];            // of the accumulators
    uint64_t scales_full[4], scales_empty[4];        // BYROW
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Fp8Ctl<7>) <= 256, "control block");

// Many rows: a pair of SMs computes 256 rows of C, as the plain product's pair does
// (gemm_kernel_2cta.cuh).  The tensor cores know no scales, so the sum over each 128 elements of
// K has an accumulator of its own, two or four of them in turn (all of TMEM), which eight warps a CTA
// multiply by the scales of its rows and columns and add to fp32 sums in registers.
//   squares: tiles of 256 columns, two accumulators, or of 128, four.  Four warps take half of the
//            columns (of one square of scales); a thread has a row, with one factor for them.  A step
//            of 128 columns is 0.25 us, of 256 it is 512 cycles
//            of the tensor cores and 128 reads of TMEM and 64 double multiply-adds of a thread: 0.40 to
//            0.43 us (2048 x 2304 x 16384, one wave of 72 pairs: 54 to 59 us, 2.6 to 2.9 PFLOP/s), 0.45 over 14
//            waves at the power limit (8192 x 8192 x 8192: 404 us), 0.34 where the MMAs do not wait for the warps.
//            Accumulators of 128 columns, 32 instead of 16 columns a read and single instead of
//            double multiply-adds all gave the same.  Nothing may spill: what is stored to local memory
//            right after its load makes the thread wait for it (0.7 to 1.2 us a step).
//   by rows: tiles of 128 columns, four accumulators.  The eight warps take 64 columns each; a thread
//            has two columns in eight of four rows, whose scales two warps bring four steps at a time
//            (read a step at a time they were 384 lines a step, more than the first-level cache
//            holds).  A step is 0.37 us; in tiles of 256 columns it was 0.73, with fewer tiles to fill the
//            SMs (1000 x 2056 x 4112: 16 us, 30 in those tiles).
template <int OUT, bool BYROW, int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_c, const Fp8Params p) {
    using L = Fp8Layout<BYROW, BN>;
    static_assert(!BYROW || BN == 128, "tiles by rows");
    constexpr int kStages = L::kStages, kTurns = L::kTurns, kBN = L::kBN, kStep = 16;
    constexpr int kTurnBits = kTurns == 4 ? 2 : 1;
    constexpr int kCols = kBN / 2;                   // of a warp
    constexpr uint32_t kPairTx = 2 * (kTileSlot + L::kBSlot);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring = smem_addr(smem), ring_b = ring + kStages * kTileSlot;
    const uint32_t staging = ring + L::kRing, scales = staging + L::kStaging + 256;
    Fp8Ctl<kStages>* ctl = reinterpret_cast<Fp8Ctl<kStages>*>(smem + L::kRing + L::kStaging);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int32_t pair = static_cast<int32_t>(blockIdx.x >> 1), npairs = static_cast<int32_t>(gridDim.x >> 1);

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmap_a);
        prefetch_tmap(&tmap_b);
        prefetch_tmap(&tmap_c);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(smem_addr(&ctl->sums_full[b]), 1);
            mbar_init(smem_addr(&ctl->sums_empty[b]), 2 * kSumWarps);   // of both CTAs
            mbar_init(smem_addr(&ctl->scales_full[b]), 64);
            mbar_init(smem_addr(&ctl->scales_empty[b]), kSumWarps);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&ctl->tmem_base), kTurns * kBN);
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

    // (each warpgroup as one: the four warps of a group change their registers together)
    if (warp < kFirstSumWarp) {
        fewer_registers<kFewRegisters>();
        if (warp == 0) {
            // ------------------------------------------------ copies (both CTAs)
            if (elect_one_sync()) {
                int stage = 0, issued = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int32_t u = pair; ok && u < p.num_units; u += npairs) {
                    int32_t m_blk, n_blk;
                    raster_tile_fast(p.m_blocks, p.rd, u, &m_blk, &n_blk);
                    const int32_t a_row = (2 * m_blk + static_cast<int32_t>(rank)) * kBM;
                    const int32_t b_row = n_blk * kBN + static_cast<int32_t>(rank) * (kBN / 2);
                    for (int32_t kb = 0; kb < p.num_kb; ++kb) {
                        if (issued >= kStages &&
                            !await(smem_addr(&ctl->empty[stage]), phase ^ 1u, watch, kSiteProducerEmpty)) {
                            ok = false;
                            break;
                        }
                        const uint32_t full = smem_addr(&ctl->full[stage]);
                        if (leader) mbar_arrive_expect_tx(full, kPairTx + p.tx_extra);
                        const uint32_t full_lead = map_to_rank(full, 0);
                        tma_load_2d_pair(ring + stage * kTileSlot, &tmap_a, full_lead, kb * kRowBytes, a_row);
                        tma_load_2d_pair(ring_b + stage * L::kBSlot, &tmap_b, full_lead, kb * kRowBytes, b_row);
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
            // ------------------------------------------------ MMAs (leader)
            if (leader && elect_one_sync()) {
                int stage = 0;
                uint32_t phase = 0, turn = 0;            // turn: steps so far
                bool ok = true;
                for (int32_t u = pair; ok && u < p.num_units; u += npairs) {
                    for (int32_t kb = 0; kb < p.num_kb; ++kb, ++turn) {
                        const uint32_t slot = turn % kTurns;
                        if (!await(smem_addr(&ctl->full[stage]), phase, watch, kSiteMmaFull) ||
                            (turn >= kTurns && !await(smem_addr(&ctl->sums_empty[slot]), ((turn >> kTurnBits) & 1u) ^ 1u, watch,
                                                           kSiteMmaTmemEmpty))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a_desc = sw128_kmajor_desc(ring + stage * kTileSlot);
                        const uint64_t b_desc = sw128_kmajor_desc(ring_b + stage * L::kBSlot);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_f8_pair(tmem_base + slot * kBN, a_desc + 2 * k, b_desc + 2 * k, p.idesc, k > 0 ? 1u : 0u);
                        umma_commit_pair(smem_addr(&ctl->sums_full[slot]), 3);
                        umma_commit_pair(smem_addr(&ctl->empty[stage]), 3);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                umma_commit_pair(smem_addr(&ctl->drain), 1);
                wait_phase_unwind(smem_addr(&ctl->drain), 0, 100000000ull);
            }
            __syncwarp();
        } else if constexpr (BYROW) {
            // ------------------------------------------------ the tile's scales, of two columns and two rows a thread
            const int first = static_cast<int>(threadIdx.x) - 64;
            uint32_t four = 0;                           // runs of four steps
            bool ok = true;
            for (int32_t u = pair; ok && u < p.num_units; u += npairs) {
                int32_t m_blk, n_blk;
                raster_tile_fast(p.m_blocks, p.rd, u, &m_blk, &n_blk);
                const int32_t row = (2 * m_blk + static_cast<int32_t>(rank)) * kBM + first, col = n_blk * kBN + first;
                const float* from[4];                    // (rows and columns outside C take the last one's)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    from[i] = i < 2 ? p.b_scales + static_cast<int64_t>(min(col + 64 * i, p.N - 1)) * p.num_kb
                                    : p.a_scales + static_cast<int64_t>(min(row + 64 * (i - 2), p.M - 1)) * p.num_kb;
                for (int32_t kb = 0; kb < p.num_kb; kb += 4, ++four) {
                    const uint32_t slot = four & 3u;
                    if (four >= 4 && !await(smem_addr(&ctl->scales_empty[slot]), ((four >> 2) & 1u) ^ 1u, watch,
                                                 kSiteProducerEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = scales + slot * L::kScaleSlot + static_cast<uint32_t>(first) * 16;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (p.whole_scales) {
                            fetch_scales(to + 64 * 16 * i, from[i] + kb);
                        } else {
                            for (int k = 0; k < 4 && kb + k < p.num_kb; ++k) fetch_scale(to + 64 * 16 * i + 4 * k, from[i] + kb + k);
                        }
                    }
                    arrive_when_fetched(smem_addr(&ctl->scales_full[slot]));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------- sums (both CTAs)
        more_registers<kSumRegisters>();
        const int quad = warp & 3, which = (warp - kFirstSumWarp) >> 2;   // which half of the columns
        const uint32_t lanes_at = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(which * kCols);
        const uint32_t buf_at = staging + static_cast<uint32_t>((warp - kFirstSumWarp) * L::kStoreBufs * L::kStoreBuf);
        uint32_t turn = 0, four = 0;                         // steps; BYROW: runs of four
        bool ok = true;
        for (int32_t u = pair; ok && u < p.num_units; u += npairs) {
            int32_t m_blk, n_blk;
            raster_tile_fast(p.m_blocks, p.rd, u, &m_blk, &n_blk);
            const int32_t y = (2 * m_blk + static_cast<int32_t>(rank)) * kBM + quad * 32;
            const int32_t x = n_blk * kBN + which * kCols;
            // 64 columns of the warp's rows, which `place` writes to a buffer of the warp.  With two buffers the
            // wait lets the newest group go on, so that has to be the other buffer's: columns behind the last
            // are a group, too, an empty one.
            const auto store = [&](int c, auto place) {
                if (y >= p.M || x + c >= p.N) {              // (the whole warp)
                    if (L::kStoreBufs > 1 && lane == 0) bulk_commit_group();
                    return;
                }
                const uint32_t buf = buf_at + static_cast<uint32_t>(c / 64 * L::kStoreBuf);
                if (lane == 0) bulk_wait_group_read<L::kStoreBufs - 1>();
                __syncwarp();
                place(buf);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tmap_c, buf, x + c, y);
                    bulk_commit_group();
                }
            };
            const auto release = [&](uint32_t slot) {        // (the accumulators are in registers)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(smem_addr(&ctl->sums_empty[slot]));
            };
            float acc[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
            if constexpr (!BYROW) {
                ScaleRow sa, sb;
                // (rows and columns outside C take the last one's scales, and are not stored)
                sa.begin(p.a_scales + static_cast<int64_t>(min(y + lane, p.M - 1)) * p.num_kb, 0);
                sb.begin(p.b_scales + static_cast<int64_t>(min(x, p.N - 1) / kTileSide) * p.num_kb, 0);
                for (int32_t kb = 0; kb < p.num_kb; ++kb, ++turn) {
                    const uint32_t slot = turn % kTurns, at = lanes_at + slot * kBN;
                    const float s = sa.get(kb + 1 < p.num_kb) * sb.get(kb + 1 < p.num_kb);
                    ok = await(smem_addr(&ctl->sums_full[slot]), (turn >> kTurnBits) & 1u, watch, kSiteEpiTmemFull);
                    if (!ok) break;
                    tc_fence_after();
                    const gbt::Pair s2(s, s);
                    uint32_t v[2][kStep];
                    tmem_read(at, v[0]);
#pragma unroll
                    for (int c = 0; c < kCols / kStep; ++c) {
                        tmem_arrived(v[c & 1]);
                        if (c + 1 < kCols / kStep) {
                            tmem_read(at + (c + 1) * kStep, v[(c + 1) & 1]);
                        } else {
                            release(slot);
                        }
#pragma unroll
                        for (int j = 0; j < kStep; j += 2) {
                            const int to = c * kStep + j;
                            const gbt::Pair t(__uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1]));
                            gbt::fma2(t, s2, gbt::Pair(acc[to], acc[to + 1])).get(acc[to], acc[to + 1]);
                        }
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < kCols; c += 64) {
                    store(c, [&](uint32_t buf) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = pack2<OUT>(acc[c + 2 * i], acc[c + 2 * i + 1]);
                        stage_store_row(buf, lane, 0, w, 8);
                    });
                }
            } else {
                const int group = lane / 4, two = lane % 4;  // rows group + 8 h, columns 8 i + 2 two, + 1
                for (int32_t kb = 0; kb < p.num_kb; ++kb, ++turn) {
                    const uint32_t slot = turn % kTurns, at = lanes_at + slot * kBN, place = four & 3u;
                    const uint32_t scales_at = scales + place * L::kScaleSlot + static_cast<uint32_t>(kb & 3) * 4;
                    if ((kb & 3) == 0)
                        ok = await(smem_addr(&ctl->scales_full[place]), (four >> 2) & 1u, watch, kSiteEpiTmemFull);
                    gbt::Pair s[4];
                    if (ok) {
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            s[h] = ld_shared_twice(scales_at + static_cast<uint32_t>(kBN + quad * 32 + 8 * h + group) * 16);
                        ok = await(smem_addr(&ctl->sums_full[slot]), (turn >> kTurnBits) & 1u, watch, kSiteEpiTmemFull);
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t cols_at = scales_at + static_cast<uint32_t>(which * kCols + 2 * two) * 16;
                    uint32_t v[2][kStep];
                    tmem_read_by_fours(at, v[0]);
                    gbt::Pair w[4];
                    // step c: columns 32 (c / 2) .. + 31 of the upper or lower 16 rows
#pragma unroll
                    for (int c = 0; c < kCols / kStep; ++c) {
                        if (c % 2 == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = ld_shared_pair(cols_at + static_cast<uint32_t>(16 * c + 8 * i) * 16);
                        }
                        tmem_arrived(v[c & 1]);
                        if (c + 1 < kCols / kStep) {
                            tmem_read_by_fours(at + ((c + 1) / 2) * 32 + (static_cast<uint32_t>((c + 1) % 2 * 16) << 16), v[(c + 1) & 1]);
                        } else {
                            release(slot);
                        }
#pragma unroll
                        for (int j = 0; j < kStep; j += 2) {
                            const int to = c * kStep + j;
                            const gbt::Pair t(__uint_as_float(v[c & 1][j]), __uint_as_float(v[c & 1][j + 1]));
                            gbt::fma2(gbt::mul2(t, w[j / 4]), s[c % 2 * 2 + j / 2 % 2], gbt::Pair(acc[to], acc[to + 1]))
                                .get(acc[to], acc[to + 1]);
                        }
                    }
                    if ((kb & 3) == 3 || kb + 1 == p.num_kb) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ctl->scales_empty[place]));
                        ++four;
                    }
                }
                if (!ok) break;
                store(0, [&](uint32_t buf) {
#pragma unroll
                    for (int c = 0; c < kCols / kStep; ++c) {
#pragma unroll
                        for (int j = 0; j < kStep; j += 2) {
                            const int r = c % 2 * 16 + j / 2 % 2 * 8 + group, unit = c / 2 * 4 + j / 4;
                            st_shared_u1(buf + static_cast<uint32_t>(r * kRowBytes + ((unit ^ (r & 7)) * 16) + two * 4),
                                         pack2<OUT>(acc[c * kStep + j], acc[c * kStep + j + 1]));
                        }
                    }
                });
            }
        }
    }

    tc_fence_before();
    cluster_sync_all();                              // the pair's MMAs, TMEM reads and copies are all finished
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTurns * kBN);
    } else if (warp >= kFirstSumWarp) {
        if (lane == 0) bulk_wait_group_read<0>();    // the stores have read their buffers
        __syncwarp();
    }
}

// ---------------------------------------------------------------- launches

template <int OUT>
bool prepare() {
    return allow_shared<fp8_pair_kernel<OUT, false, 256>>(Fp8Layout<false, 256>::kTotal) &&
           allow_shared<fp8_pair_kernel<OUT, false, 128>>(Fp8Layout<false, 128>::kTotal) &&
           allow_shared<fp8_pair_kernel<OUT, true, 128>>(Fp8Layout<true, 128>::kTotal) &&
           allow_shared<few_rows_kernel<true, OUT, 32>>(FewLayout<32>::kTotal) &&
           allow_shared<few_rows_kernel<true, OUT, 128>>(FewLayout<128>::kTotal);
}

// The kernel and, by squares, its tiles' columns: a step of 128 takes 0.6 of one of 256, so they are taken
// where they make less than 1.6 times the waves (512 x 4096 x 4096: 64 tiles or 32 for 76 pairs, 11.3 and
// 16.0 us; 1024 x 4096 x 4096: 128 or 64, 19.3 and 17.1; 8192 x 8192 x 8192: 465 and 405).
void choose(gemm_fp8_plan* p) {
    constexpr FewRates kRates{0.29, 0.33, 1.6, 0.38, 0.5};
    p->choice = FewChoice{0, 0};
    p->width = 128;
    if (p->b_scales != GEMM_SCALE_SQUARE) return;
    const int64_t pairs = p->base.num_sms / 2, m_blocks = (p->M + 255) / 256;
    const auto waves = [&](int64_t width) { return (m_blocks * ((p->N + width - 1) / width) + pairs - 1) / pairs; };
    const double wide = static_cast<double>(waves(256)), narrow = 0.6 * static_cast<double>(waves(128));
    if (narrow >= wide) p->width = 256;
    p->choice = choose_kernel(p->M, gbt::groups_of(p->M) * gbt::groups_of(p->N), p->width == 256 ? wide : narrow,
                              static_cast<int>(gbt::groups_of(p->K)), static_cast<double>(p->N) * p->K, p->base.num_sms, kRates);
}

template <int OUT>
gemm_status_t run(const gemm_fp8_plan* p, const void* A, const float* a_scales, const void* B, const float* b_scales, void* C,
                  gbt::Queue queue) {
    const int64_t M = p->M, N = p->N, K = p->K;
    const int32_t num_kb = static_cast<int32_t>(gbt::groups_of(K));
    const int64_t few_tiles = gbt::groups_of(M) * gbt::groups_of(N);
    const FewChoice& choice = p->choice;
    const bool few = choice.slices > 0;
    const int box = few && M <= 32 ? 32 : kTileSide;
    CUtensorMap a, b, c;
    if (!encode_map(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, A, M, K, K, box) ||
        !encode_map(&b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, B, N, K, K, few ? kTileSide : p->width / 2))
        return GEMM_ERR_TENSORMAP;
    if (few) {
        FewParams f{};
        f.M = static_cast<int32_t>(M);
        f.N = static_cast<int32_t>(N);
        f.num_kb = num_kb;
        f.m_blocks = static_cast<int32_t>(gbt::groups_of(M));
        f.slices = choice.slices;
        f.kb_per_slice = choice.kb_per_slice;
        f.idesc = descriptor(0, kTileSide, kTileSide);
        f.tx_extra = p->base.tx_extra;
        f.a_scales = a_scales;
        f.b_scales = b_scales;
        f.out = C;
        f.error_word = p->base.error_word;
        f.timeout_ns = p->base.timeout_ns;
        if (box == 32)
            return gbt::launch<few_rows_kernel<true, OUT, 32>>(few_tiles * f.slices, kThreads, FewLayout<32>::kTotal, queue, f.slices, a,
                                                               b, b, f);
        return gbt::launch<few_rows_kernel<true, OUT, 128>>(few_tiles * f.slices, kThreads, FewLayout<128>::kTotal, queue, f.slices, a, b,
                                                            b, f);
    }
    if (!encode_map(&c, OUT == kOutF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, C, M, N, N, 32))
        return GEMM_ERR_TENSORMAP;
    Fp8Params f{};
    f.M = static_cast<int32_t>(M);
    f.N = static_cast<int32_t>(N);
    f.num_kb = num_kb;
    f.m_blocks = static_cast<int32_t>((M + 255) / 256);
    const int32_t n_blocks = static_cast<int32_t>((N + p->width - 1) / p->width);
    f.num_units = f.m_blocks * n_blocks;
    f.idesc = descriptor(0, 256, p->width);
    f.tx_extra = p->base.tx_extra;
    f.whole_scales = num_kb % 4 == 0 && gbt::aligned(a_scales, 16) && gbt::aligned(b_scales, 16);
    f.a_scales = a_scales;
    f.b_scales = b_scales;
    f.error_word = p->base.error_word;
    f.timeout_ns = p->base.timeout_ns;
    // bands of eight row blocks: the 76 pairs cover about 8 x 9 tiles at a time
    f.rd = make_raster_div(f.m_blocks, n_blocks, f.m_blocks < 8 ? f.m_blocks : 8);
    const int pairs = p->base.num_sms / 2, grid = 2 * (f.num_units < pairs ? f.num_units : pairs);
    const auto go = [&](auto byrow, auto width) {
        constexpr bool kByRow = decltype(byrow)::value;
        constexpr int kWidth = decltype(width)::value;
        return gbt::launch<fp8_pair_kernel<OUT, kByRow, kWidth>>(grid, kPairThreads, Fp8Layout<kByRow, kWidth>::kTotal, queue, 2, a, b,
                                                                 c, f);
    };
    if (p->b_scales == GEMM_SCALE_ROW) return go(std::true_type(), std::integral_constant<int, 128>());
    return p->width == 128 ? go(std::false_type(), std::integral_constant<int, 128>())
                           : go(std::false_type(), std::integral_constant<int, 256>());
}

}  // namespace
}  // namespace gbf

extern "C" {

gemm_status_t gemm_fp8_plan_create(int64_t M, int64_t N, int64_t K, gemm_elem_t out, gemm_scale_t b_scales,
                                   gemm_fp8_plan_t* plan) {
    using namespace gbf;
    if (!plan) return GEMM_ERR_INVALID_ARG;
    *plan = nullptr;
    if ((out != GEMM_ELEM_F16 && out != GEMM_ELEM_BF16) || (b_scales != GEMM_SCALE_ROW && b_scales != GEMM_SCALE_SQUARE))
        return GEMM_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0 || M > INT32_MAX - 256 || N > INT32_MAX - 256 || K > INT32_MAX - 128) return GEMM_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 16 != 0) return GEMM_ERR_ALIGNMENT;
    if ((M / 128 + 1) * (N / 128 + 1) > (int64_t{1} << 27)) return GEMM_ERR_INVALID_ARG;   // tiles in 32 bits
    gemm_fp8_plan* p = new (std::nothrow) gemm_fp8_plan();
    if (!p) return GEMM_ERR_OOM;
    p->M = M;
    p->N = N;
    p->K = K;
    p->out = out;
    p->b_scales = b_scales;
    gemm_status_t st = open_plan(&p->base);
    if (st == GEMM_OK && !(out == GEMM_ELEM_F16 ? prepare<kOutF16>() : prepare<kOutBF16>())) {
        close_plan(&p->base);
        st = GEMM_ERR_LAUNCH;
    }
    if (st != GEMM_OK) {
        delete p;
        return st;
    }
    choose(p);
    *plan = p;
    return GEMM_OK;
}

gemm_status_t gemm_fp8_run(gemm_fp8_plan_t p, const void* A, const float* a_scales, const void* B, const float* b_scales,
                           void* C, void* stream) {
    using namespace gbf;
    if (!p) return GEMM_ERR_INVALID_ARG;
    const gemm_status_t st = gbt::check_device(p->base.device);
    if (st != GEMM_OK) return st;
    if (p->M == 0 || p->N == 0) return GEMM_OK;
    if (!C || (p->K > 0 && (!A || !B || !a_scales || !b_scales))) return GEMM_ERR_INVALID_ARG;
    if (!gbt::aligned(A, 16) || !gbt::aligned(B, 16) || !gbt::aligned(C, 16) || !gbt::aligned(a_scales, 4) ||
        !gbt::aligned(b_scales, 4))
        return GEMM_ERR_ALIGNMENT;
    if (p->K == 0) {
        if (launch_zero_fill(C, p->M * p->N * 2, p->base.num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess)
            return GEMM_OK;
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    const gbt::Queue queue{stream, p->base.device};
    return p->out == GEMM_ELEM_F16 ? run<kOutF16>(p, A, a_scales, B, b_scales, C, queue)
                                   : run<kOutBF16>(p, A, a_scales, B, b_scales, C, queue);
}

gemm_status_t gemm_fp8_plan_set_timeout(gemm_fp8_plan_t p, uint64_t ns) {
    if (!p) return GEMM_ERR_INVALID_ARG;
    p->base.timeout_ns = ns ? ns : gbf::kWaitLimitNs;
    return GEMM_OK;
}

gemm_status_t gemm_fp8_plan_set_wait_test(gemm_fp8_plan_t p, uint32_t extra_bytes) {
    if (!p || extra_bytes > 4096 || (extra_bytes & 15u)) return GEMM_ERR_INVALID_ARG;
    p->base.tx_extra = extra_bytes;
    return GEMM_OK;
}

gemm_status_t gemm_fp8_plan_check(gemm_fp8_plan_t p, void* stream) {
    return p ? gbf::check_plan(&p->base, stream) : GEMM_ERR_INVALID_ARG;
}

gemm_status_t gemm_fp8_plan_destroy(gemm_fp8_plan_t p) {
    if (!p) return GEMM_OK;
    const gemm_status_t st = gbf::close_plan(&p->base);
    delete p;
    return st;
}

}  // extern "C"
