// ffn_mma.cuh -- what the gated and the 8-bit product share: the product of few rows over a
// cluster's slices of K, tensor maps and the plan's launch parts.
//
// The conventions are those of gemm_kernel.cuh (whose PTX wrappers are used): a producer warp
// fills a ring by TMA, one thread issues tcgen05.mma into TMEM, epilogue warps take the sums
// from there; every wait is bounded and leads to the common exit when it runs out.
#pragma once
#include <cmath>

#include "ffn_common.cuh"
#include "gemm_kernel_2cta.cuh"

namespace gbf {

using namespace gbg;

constexpr int kRowBytes = 128;                       // of one k-block of an operand's row: a swizzle span
constexpr int kTileSide = 128;                       // rows of a CTA's tile, and of an operand's box
constexpr int kTileSlot = kTileSide * kRowBytes;     // 16 KiB

// The accumulators that a tcgen05.ld brought are there (tied to the registers, so that no use of
// them can be moved before the wait).
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}
// 32 lanes x 16 or 8 consecutive 32-bit TMEM columns -> as many registers per thread.
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :: "memory");
}
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// 16 lanes x 32 consecutive TMEM columns -> 16 registers per thread: for i < 4, registers 4i, 4i + 1 are
// columns 8i + 2 (t % 4), + 1 of lane t / 4, and 4i + 2, 4i + 3 those of lane t / 4 + 8.
__device__ __forceinline__ void tmem_read_by_fours(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// The registers of a warpgroup (all of its warps): fewer, or more out of what others gave up.
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One K = 32 step over e4m3 operands.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// As wait_phase, which reads the global timer once the first look has failed; here only after many.
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, const Watch& w, int32_t site) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_phase(bar, parity, w, site);
}

// sigmoid(g), relative to its value on both sides of zero: within 3.5e-7 for g from -4 up, then with __expf's error,
// which grows with the argument (1e-6 at -20, 4e-6 at -80; from -87 down its results leave the normal range).
__device__ __forceinline__ float sigmoid(float g) {
    const float e = __expf(-fabsf(g));
    const float s = __fdividef(1.f, 1.f + e);
    return g < 0.f ? e * s : s;
}
// exp(-g^2 / 2)
__device__ __forceinline__ float bell(float g) {
    const float w = g * 0.84932180f;                  // sqrt(log2(e) / 2)
    return gbt::exp2_fast(-(w * w));
}
// The normal distribution's Phi(g), both tails to relative accuracy, with e = bell(g).  For z =
// |g| / sqrt 2 the upper tail is erfc(z) / 2 = exp(-z^2) t Q(t) / 2 with t = 1 / (1 + 0.45 z): a smooth
// function of t in (0, 1], here a polynomial of degree 7 fitted to erfc(z) exp(z^2) / t for z up to 10
// (weighted least squares, the weights moved to the largest relative errors; 3.1e-7 at most).
// With the exponential's rounding the lower tail is within 1.2e-6 for |g| up to 4, 5.2e-6 up to 8 and 1.3e-5 at 13
// (below 2^-126 it is zero), which 16-bit results do not show.  erfcf took 6 us more of
// 1024 x 4096 x 2048 (23 us with SiLU).
__device__ __forceinline__ float normal_cdf(float g, float e) {
    const float t = __fdividef(1.f, fmaf(0.45f * 0.70710678f, fabsf(g), 1.f));
    float q = fmaf(6.684802473e-02f, t, -2.401618809e-01f);
    q = fmaf(q, t, 2.086041719e-01f);
    q = fmaf(q, t, 4.054885730e-02f);
    q = fmaf(q, t, 1.884976625e-01f);
    q = fmaf(q, t, 2.281251252e-01f);
    q = fmaf(q, t, 2.536289692e-01f);
    q = fmaf(q, t, 2.539093792e-01f);
    q *= 0.5f * t * e;
    return g < 0.f ? q : 1.f - q;
}
// act(g) of gemm_activation_t, with the lower tails relative to their values (see above).
template <int ACT>
__device__ __forceinline__ float gate_fn(float g) {
    if constexpr (ACT == GEMM_ACT_RELU) return fmaxf(g, 0.f) + (g != g ? g : 0.f);
    if constexpr (ACT == GEMM_ACT_GELU) return g * normal_cdf(g, bell(g));
    if constexpr (ACT == GEMM_ACT_SILU) return g * sigmoid(g);
    return g;
}
// Calls f with act as a compile-time value.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case GEMM_ACT_RELU: f(std::integral_constant<int, GEMM_ACT_RELU>()); break;
        case GEMM_ACT_GELU: f(std::integral_constant<int, GEMM_ACT_GELU>()); break;
        case GEMM_ACT_SILU: f(std::integral_constant<int, GEMM_ACT_SILU>()); break;
        default: f(std::integral_constant<int, GEMM_ACT_NONE>()); break;
    }
}

// ---- scales along K -------------------------------------------------------------------

// One row of scales, each read a step before its use.  (A thread's reads of 32 groups are one
// line; four at a time took registers that the sums need.  The read is volatile to stay
// before the wait that hides it: left to the compiler it moved to its use.)
struct ScaleRow {
    const float* at;
    float next;
    __device__ __forceinline__ void read() { asm volatile("ld.global.f32 %0, [%1];" : "=f"(next) : "l"(at)); }
    __device__ __forceinline__ void begin(const float* row, int kb) {
        at = row + kb;
        read();
    }
    __device__ __forceinline__ float get(bool more) {
        const float now = next;
        ++at;
        if (more) read();
        return now;
    }
};

// Arrive on the pair leader's barrier at this offset.  (What it orders are reads of TMEM, which
// are complete: a release at cluster scope would wait for every load in flight besides, and
// took two thirds of the 8-bit product's time.)
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, 0)) : "memory");
}

// ---- few rows: one tile of up to 128 rows by 128 weight rows a cluster, K in slices -----------
//
// Few rows are bound by the weights' bytes, so all SMs have to stream them: the S CTAs of a
// cluster (1, 2, 4 or 8) take the k-blocks of one tile in S runs, and add their sums through
// distributed shared memory in the order of the runs.  About 100 KiB of ring a CTA: two
// share an SM, and one streams while the other starts or ends.  Of the rows (the MMA's
// M = 128) only RM are copied; the MMA reads what lies behind them in the ring for the others,
// which are never looked at.
//   gated: weight rows f .. f+63 of the gate and of the other half, side by side in N; 16-bit
//          operands, one accumulator over the run
//   8 bit: 128 rows of B; an accumulator for each 128 elements of K (two in turn), multiplied by
//          its scales into registers

struct FewParams {
    int32_t M, N;                // rows; columns of the result
    int32_t num_kb, m_blocks, slices, kb_per_slice;
    uint32_t idesc, tx_extra;
    int32_t act;                 // gated
    const float* a_scales;
    const float* b_scales;
    void* out;                   // M x N
    void* gate_up;               // gated: M x 2N, or NULL
    int32_t* error_word;
    uint64_t timeout_ns;
};

template <int RM>
struct FewLayout {
    static constexpr int kStages = RM == 32 ? 5 : 3;
    static constexpr int kASlot = RM * kRowBytes;
    static constexpr int kRing = kStages * (kASlot + kTileSlot);
    static constexpr int kTotal = 1024 + kRing + 256;
    static_assert((kStages - 1) * kASlot + kTileSlot <= kRing, "the MMA's rows stay within the ring");
    static_assert(RM * kTileSide * 4 <= kRing, "sums are exchanged in the ring");
    static_assert(2 * (kTotal + 1024) <= 233472, "two CTAs share an SM");
};

// Offset of four sums (columns 4 c4 ..) of a row: units exchanged so that the rows of a warp
// write to distinct banks.
__device__ __forceinline__ uint32_t sums_at(int row, int c4) {
    return static_cast<uint32_t>(row * kTileSide * 4 + ((c4 ^ (row & 31)) * 16));
}

// The end of a tile whose S slices' sums stand in their CTAs' shared memory: each CTA finishes every
// S-th run of groups of four columns.  All slices' loads are under way before the first is
// used: one way to the other SMs, not S.
template <bool F8, int OUT, int RM, int S>
__device__ __forceinline__ void few_rows_finish(const FewParams& p, uint32_t sums, int row0, int n_blk, int slice) {
    constexpr int kAcross = F8 ? kTileSide / 4 : kTileSide / 8;
    const int rows = min(RM, p.M - row0), groups = rows * kAcross;
    const int col0 = n_blk * (F8 ? kTileSide : kTileSide / 2);
    uint32_t base[S];
#pragma unroll
    for (int s = 0; s < S; ++s) base[s] = map_to_rank(sums, static_cast<uint32_t>(s));
    for (int i = slice * kThreads + static_cast<int>(threadIdx.x); i < groups; i += S * kThreads) {
        const int row = i / kAcross, c4 = i % kAcross, col = col0 + c4 * 4;
        if (col >= p.N) continue;                        // (N % 8 == 0)
        const uint32_t at = sums_at(row, c4), at_u = sums_at(row, (c4 + kAcross) % (kTileSide / 4));
        uint4 v[S], w[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            v[s] = ld_dsmem_u4(base[s] + at);
            if constexpr (!F8) w[s] = ld_dsmem_u4(base[s] + at_u);
        }
        float g[4] = {}, u[4] = {};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            g[0] += __uint_as_float(v[s].x);
            g[1] += __uint_as_float(v[s].y);
            g[2] += __uint_as_float(v[s].z);
            g[3] += __uint_as_float(v[s].w);
            if constexpr (!F8) {
                u[0] += __uint_as_float(w[s].x);
                u[1] += __uint_as_float(w[s].y);
                u[2] += __uint_as_float(w[s].z);
                u[3] += __uint_as_float(w[s].w);
            }
        }
        if constexpr (!F8) {
            if (p.gate_up) {
                uint16_t* to = static_cast<uint16_t*>(p.gate_up) + static_cast<int64_t>(row0 + row) * 2 * p.N + col;
                *reinterpret_cast<uint2*>(to) = make_uint2(pack2<OUT>(g[0], g[1]), pack2<OUT>(g[2], g[3]));
                *reinterpret_cast<uint2*>(to + p.N) = make_uint2(pack2<OUT>(u[0], u[1]), pack2<OUT>(u[2], u[3]));
            }
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int k = 0; k < 4; ++k) g[k] = gate_fn<decltype(act)::value>(g[k]) * u[k];
            });
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(row0 + row) * p.N + col) =
            make_uint2(pack2<OUT>(g[0], g[1]), pack2<OUT>(g[2], g[3]));
    }
}

// All threads of the cluster have come here; orders no memory (a release would wait for the results'
// stores to be performed).
__device__ __forceinline__ void leave_together() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

template <bool F8, int OUT, int RM>
__global__ void __launch_bounds__(kThreads, 2)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                    const __grid_constant__ CUtensorMap tmap_b2, const FewParams p) {
    using L = FewLayout<RM>;
    constexpr int kStages = L::kStages;
    constexpr int kWarps = RM / 32;                       // epilogue warps that hold rows
    constexpr uint32_t kTmemCols = F8 ? 256 : 128;
    constexpr uint32_t kTx = L::kASlot + kTileSlot;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t ring_a = smem_addr(smem), ring_b = ring_a + kStages * L::kASlot;
    SharedCtl<kStages>* ctl = reinterpret_cast<SharedCtl<kStages>*>(smem + L::kRing);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int slice = static_cast<int>(cluster_ctarank());
    const int unit = static_cast<int>(blockIdx.x) / p.slices;
    const int n_blk = unit / p.m_blocks, m_blk = unit - n_blk * p.m_blocks;
    const int kb0 = min(slice * p.kb_per_slice, p.num_kb), kb1 = min(kb0 + p.kb_per_slice, p.num_kb);
    const int row0 = m_blk * kTileSide;
    constexpr int kElems = F8 ? kRowBytes : kRowBytes / 2;  // of a k-block

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmap_a);
        prefetch_tmap(&tmap_b);
        if (!F8) prefetch_tmap(&tmap_b2);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&ctl->full[s]), 1);
            mbar_init(smem_addr(&ctl->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&ctl->tmem_full[b]), 1);
            mbar_init(smem_addr(&ctl->tmem_empty[b]), kWarps);
        }
        mbar_init(smem_addr(&ctl->drain), 1);
        ctl->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&ctl->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const Watch watch{&ctl->abort, p.error_word, p.timeout_ns};
    if (warp == 0 && elect_one_sync()) {
        // the first weights on their way to the second-level cache while the previous kernel ends
        for (int kb = kb0; kb < kb1 && kb < kb0 + kStages; ++kb) {
            if constexpr (F8) {
                tma_prefetch_l2_2d(&tmap_b, kb * kElems, n_blk * kTileSide);
            } else {
                tma_prefetch_l2_2d(&tmap_b, kb * kElems, n_blk * (kTileSide / 2));
                tma_prefetch_l2_2d(&tmap_b2, kb * kElems, n_blk * (kTileSide / 2));
            }
        }
    }
    __syncwarp();
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == 0) {
        if (elect_one_sync()) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (issued >= kStages &&
                    !wait_phase(smem_addr(&ctl->empty[stage]), phase ^ 1u, watch, kSiteProducerEmpty))
                    break;
                const uint32_t full = smem_addr(&ctl->full[stage]);
                mbar_arrive_expect_tx(full, kTx + p.tx_extra);
                const uint32_t b_slot = ring_b + stage * kTileSlot;
                if constexpr (F8) {
                    tma_load_2d(b_slot, &tmap_b, full, kb * kElems, n_blk * kTileSide);
                } else {
                    tma_load_2d(b_slot, &tmap_b, full, kb * kElems, n_blk * (kTileSide / 2));
                    tma_load_2d(b_slot + kTileSlot / 2, &tmap_b2, full, kb * kElems, n_blk * (kTileSide / 2));
                }
                tma_load_2d(ring_a + stage * L::kASlot, &tmap_a, full, kb * kElems, row0);
                ++issued;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // what was asked for lands before the CTA can leave (at once, in normal operation)
            const int pending = issued < kStages ? issued : kStages;
            for (int i = 0; i < pending; ++i) {
                if (--stage < 0) {
                    stage = kStages - 1;
                    phase ^= 1u;
                }
                wait_phase_unwind(smem_addr(&ctl->full[stage]), phase, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one_sync()) {
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const uint32_t i = static_cast<uint32_t>(kb - kb0), buf = F8 ? i & 1u : 0u;
                if (F8 && i >= 2 &&
                    !wait_phase(smem_addr(&ctl->tmem_empty[buf]), ((i >> 1) & 1u) ^ 1u, watch, kSiteMmaTmemEmpty))
                    break;
                if (!wait_phase(smem_addr(&ctl->full[stage]), phase, watch, kSiteMmaFull)) break;
                tc_fence_after();
                const uint64_t a_desc = sw128_kmajor_desc(ring_a + stage * L::kASlot);
                const uint64_t b_desc = sw128_kmajor_desc(ring_b + stage * kTileSlot);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (F8) {
                        umma_f8(tmem_base + buf * kTileSide, a_desc + 2 * k, b_desc + 2 * k, p.idesc, k > 0 ? 1u : 0u);
                    } else {
                        umma_f16(tmem_base, a_desc + 2 * k, b_desc + 2 * k, p.idesc, kb > kb0 || k > 0 ? 1u : 0u);
                    }
                }
                umma_commit(smem_addr(&ctl->empty[stage]));
                if (F8 || kb + 1 == kb1) umma_commit(smem_addr(&ctl->tmem_full[buf]));
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            umma_commit(smem_addr(&ctl->drain));
            wait_phase_unwind(smem_addr(&ctl->drain), 0, 100000000ull);
        }
        __syncwarp();
    } else if ((warp & 3) < kWarps) {
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes_at = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        bool ok = kb0 < kb1;
        if constexpr (F8) {
            float acc[kTileSide];
#pragma unroll
            for (int c = 0; c < kTileSide; ++c) acc[c] = 0.f;
            ScaleRow sa, sb;
            if (ok) {                                    // (rows behind the last take its scales, and are not stored)
                sa.begin(p.a_scales + static_cast<int64_t>(min(row0 + row, p.M - 1)) * p.num_kb, kb0);
                sb.begin(p.b_scales + static_cast<int64_t>(n_blk) * p.num_kb, kb0);
            }
            for (int kb = kb0; kb < kb1; ++kb) {
                const uint32_t i = static_cast<uint32_t>(kb - kb0), buf = i & 1u;
                const float s = sa.get(kb + 1 < kb1) * sb.get(kb + 1 < kb1);
                if (!wait_phase(smem_addr(&ctl->tmem_full[buf]), (i >> 1) & 1u, watch, kSiteEpiTmemFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const gbt::Pair s2(s, s);
                uint32_t v[2][8];
                tmem_read(lanes_at + buf * kTileSide, v[0]);
#pragma unroll
                for (int c = 0; c < kTileSide / 8; ++c) {
                    tmem_arrived(v[c & 1]);
                    if (c + 1 < kTileSide / 8) {
                        tmem_read(lanes_at + buf * kTileSide + (c + 1) * 8, v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ctl->tmem_empty[buf]));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = c * 8 + 2 * j;
                        const gbt::Pair t(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1]));
                        gbt::fma2(t, s2, gbt::Pair(acc[at], acc[at + 1])).get(acc[at], acc[at + 1]);
                    }
                }
            }
            fence_proxy_async_smem();
            if (ok || kb0 == kb1) {
#pragma unroll
                for (int c = 0; c < kTileSide / 4; ++c)
                    st_shared_u4(ring_a + sums_at(row, c),
                                 make_uint4(__float_as_uint(acc[4 * c]), __float_as_uint(acc[4 * c + 1]),
                                            __float_as_uint(acc[4 * c + 2]), __float_as_uint(acc[4 * c + 3])));
            }
        } else {
            if (ok) ok = wait_phase(smem_addr(&ctl->tmem_full[0]), 0, watch, kSiteEpiTmemFull);
            tc_fence_after();
            fence_proxy_async_smem();
#pragma unroll
            for (int c = 0; c < kTileSide / 32; ++c) {
                uint32_t v[32];
                if (ok) {
                    tmem_ld_32x32b_x32(lanes_at + c * 32, v);
                    tmem_ld_wait();
                } else if (kb0 == kb1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                } else {
                    break;                               // (a wait ran out: copies may still land in the ring)
                }
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    st_shared_u4(ring_a + sums_at(row, c * 8 + g),
                                 make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]));
            }
        }
    }
    tc_fence_before();
    if (p.slices > 1) {
        cluster_sync_all();                              // the slices' sums are there
    } else {
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);

    switch (p.slices) {
        case 1: few_rows_finish<F8, OUT, RM, 1>(p, ring_a, row0, n_blk, slice); break;
        case 2: few_rows_finish<F8, OUT, RM, 2>(p, ring_a, row0, n_blk, slice); break;
        case 4: few_rows_finish<F8, OUT, RM, 4>(p, ring_a, row0, n_blk, slice); break;
        default: few_rows_finish<F8, OUT, RM, 8>(p, ring_a, row0, n_blk, slice); break;
    }
    if (p.slices > 1) leave_together();                  // (nobody reads this CTA's sums any more)
}

// ---- host -----------------------------------------------------------------------------

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A map over a row-major matrix whose boxes are 128 bytes of `box_rows` rows, 128-byte swizzled;
// outside the matrix zeros are read and nothing is written.
inline bool encode_map(CUtensorMap* map, CUtensorMapDataType type, int bytes, const void* base, int64_t rows, int64_t cols,
                       int64_t stride, int box_rows) {
    if (!map_encoder()) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * bytes};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kRowBytes / bytes), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t steps[2] = {1, 1};
    return map_encoder()(map, type, 2, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tcgen05 instruction descriptor: fp32 sums, both operands K-major.
constexpr uint32_t descriptor(uint32_t format, int m, int n) {
    return (1u << 4) | (format << 7) | (format << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

template <auto Kernel>
bool allow_shared(int bytes) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;

// What a plan keeps beside its shape: the device, the error word and the waits' settings.
struct PlanBase {
    int device, num_sms;
    int32_t* error_word;
    uint64_t timeout_ns;
    uint32_t tx_extra;
};

inline gemm_status_t open_plan(PlanBase* b) {
    gemm_status_t st = gbt::begin_plan(&b->device, &b->num_sms);
    if (st != GEMM_OK) return st;
    void* word = nullptr;
    st = gbt::allocate(&word, 256);
    if (st == GEMM_OK && gbt::clear_now(word, 256) != GEMM_OK) {
        cudaFree(word);
        return GEMM_ERR_CUDA;
    }
    b->error_word = static_cast<int32_t*>(word);
    b->timeout_ns = kWaitLimitNs;
    b->tx_extra = 0;
    return st;
}

inline gemm_status_t close_plan(PlanBase* b) {
    if (cudaFree(b->error_word) == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_CUDA;
}

// GEMM_ERR_DEVICE_TIMEOUT if a wait ran out since the last check.
inline gemm_status_t check_plan(PlanBase* b, void* stream) {
    const gemm_status_t st = gbt::check_error_word(b->error_word, stream);
    return st == GEMM_ERR_INDEX ? GEMM_ERR_DEVICE_TIMEOUT : st;   // (any site code is a wait's)
}

// ---- which kernel: estimates in microseconds, from measurements between 1 and 1024 rows of weights from
// 1024 x 512 to 16384 x 8192 (within a quarter of the measured time where the choice is close)

struct FewRates {
    double kb_32, kb_128;       // a k-block of a CTA whose SM it has alone, for boxes of 32 and of 128 rows
    double shared;              // ... times this where two share the SM
    double pair_kb, pair_wave;  // a k-block, and a tile's end, of the kernel of many rows
};
struct FewChoice {
    int slices;                 // of K, of the kernel of few rows; 0: the kernel of many rows is faster
    int kb_per_slice;
};

// few_tiles: tiles of the kernel of few rows; pair_waves: waves of the other one's over the pairs of SMs;
// weight_bytes: what has to come from memory in any case.  Up to 128 rows the kernel of few rows takes
// all: both are bound by memory there, and the other one streams worse (1 x 8192 x 4096 gated 40 against
// 24 us, 128 rows 27 against 27).
inline FewChoice choose_kernel(int64_t rows, int64_t few_tiles, double pair_waves, int num_kb, double weight_bytes, int num_sms,
                               const FewRates& r) {
    // (the weights' way from memory and the rest overlap, less the nearer they are to each other)
    const double memory = 2.2 + weight_bytes / 6.6e6;
    const auto with_memory = [&](double time) { return std::sqrt(std::sqrt(time * time * time * time + memory * memory * memory * memory)); };
    FewChoice best{0, 0};
    double least = 0;
    const bool few_only = rows <= kTileSide;
    if (!few_only) least = with_memory(3 + pair_waves * (num_kb * r.pair_kb + r.pair_wave));
    // CTAs of a cluster of s that are resident at once, two an SM: clusters of eight do not fill the
    // GPU's groups of SMs (15 clusters of 152 SMs with one CTA each, 36 of four)
    const double resident[] = {2.0, 2.0, 1.89, 1.57};
    for (int s = 1, k = 0; s <= 8 && s <= num_kb; s *= 2, ++k) {
        const int per = (num_kb + s - 1) / s;
        const int64_t ctas = few_tiles * s, slots = static_cast<int64_t>(resident[k] * num_sms);
        const int64_t waves = (ctas + slots - 1) / slots;
        const double kb = (rows <= 32 ? r.kb_32 : r.kb_128) * (ctas > num_sms ? r.shared : 1.0);
        // (each further wave starts its CTAs anew: 5632 x 11264 x 64 gated, 26 waves of one k-block, takes 114 us)
        const double time = with_memory(2 + 0.7 * k + static_cast<double>(waves) * (per * kb + (s > 1 ? 1.0 : 0.5)) +
                                        3.4 * static_cast<double>(waves - 1));
        if ((best.slices == 0 && few_only) || time < least) {
            best = FewChoice{s, per};
            least = time;
        }
    }
    return best;
}

}  // namespace gbf
