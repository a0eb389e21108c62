// Products of microscaled 4-bit matrices on sm_100a tensor cores: D = A B^T with A and B
// K-major e2m1 codes, a scale for each block of 16 (e4m3) or 32 (e8m0) of K on both
// sides, fp32 accumulation in tensor memory (tcgen05.mma, block-scaled kinds).
//
// Y[M, N] = X W^T takes one of three kernels: up to 16 tokens a cluster per 128 weight rows
// (k_decode_fp4), up to 128 tokens a CTA per 128 weight rows (k_gemm_fp4: the tile is as
// narrow as the tokens, and the call streams the weights once), and beyond that CTA pairs
// (k_gemm2_fp4), whose 256 x 256 tiles reuse what they read.  Measured with the packing of
// X (nv, graph replays): 1 token of 11008 x 4096 7.7 us (3.3 TB/s of packed weights), 64 tokens
// 11.9 us, 128 tokens 13.1 us, 1 token of 28672 x 8192 27 us (4.9 TB/s); 4096 tokens of 11008 x 4096
// 91 us (4.05 PFLOP/s), 8192^3 236 us (4.65; mx 214 us, 5.15).  The large ones are of a few
// dozen calls, during which the SM clock stays at 1965 MHz; when calls on random data go on
// for tens of milliseconds the power cap takes it to 1650 MHz, and the 4096 tokens take 105 us
// (mx 84 and 97).
//
// k_gemm_fp4: a CTA makes one 128 x NT tile of W X^T.  A producer thread brings stages of 256 K values: the
// code tiles by TMA (128 bytes of K per row, 128-byte swizzle) and the scale tiles by
// bulk copies.  The issuing thread copies a stage's scale tiles from shared to tensor
// memory (tcgen05.cp, ordered before the MMAs that read them) and issues one MMA per 64
// values of K.  Each ring slot has its own scale columns in tensor memory, so that the
// barrier that frees the slot's shared memory frees them too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "eqat_fp4.cuh"
#include "eqat_internal.h"
#include "eqat_pdl.cuh"
#include "eqat_ptx.cuh"
#include "eqat_qmath.cuh"

namespace eqat {
namespace {

constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr int kKStage = 256;         // K values per stage: 128 bytes of codes per row
constexpr int kSfTile = 512;         // bytes of a scale tile: 128 rows x 4 blocks
constexpr int kATile = 128 * 128;    // bytes of A per stage
constexpr int kThreads = 192;        // producer, issuer, four epilogue warps
constexpr int kHalfSmem = 113 * 1024;  // two CTAs on an SM: shared memory and
constexpr int kHalfTmem = 256;         // tensor-memory columns of each

// DEEP: a CTA has its SM for itself; otherwise two share it.
template <int NT, bool NV, bool DEEP>
struct Cfg {
    static constexpr int SF = NV ? 4 : 2;              // scale tiles of a stage per 128 rows
    static constexpr int KSF = NV ? 64 : 128;          // K values of a scale tile
    static constexpr int BTILE = NT * 128;
    static constexpr int STAGE = kATile + BTILE + 2 * SF * kSfTile;
    static constexpr int FIT = ((DEEP ? 232448 : kHalfSmem) - 1280) / STAGE;
    static constexpr int STAGES = FIT < 8 ? FIT : 8;   // 6 to 8 deep, 3 to 5
    static constexpr int TMEM = DEEP ? 512 : kHalfTmem;
    static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
    static constexpr int PART = 128 * NT * 4;          // a CTA's part of the sums, in the stages' place
    static constexpr int ACC = NT < 32 ? 32 : NT;      // accumulator columns
    static constexpr int SF_COLS = 2 * SF * 4;         // scale columns of a stage
    static_assert(NT <= 128, "one scale tile covers the rows of B");
    static_assert(ACC + STAGES * SF_COLS <= TMEM, "tensor memory columns");
    static_assert(STAGES >= 3 && PART <= STAGES * STAGE, "shared memory");
    static_assert(STAGE % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

struct Ctl {
    uint64_t full[8], empty[8], acc_full, drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Ctl) <= 256, "control block exceeds its slot");

struct Args {
    const uint8_t *sfa, *sfb;   // scale tiles
    int64_t sf_tiles_k;         // scale tiles along K (the same on both sides)
    int64_t rows_a, rows_b;     // rows of A and B
    int K;
    const float *ga, *gb;       // tensor scales (nullable)
    __nv_bfloat16 *Y;           // [rows_b, rows_a]
    int ranks;                  // CTAs of a cluster, which split K
    int *err;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Copies one scale tile (32 rows of 16 bytes) to four tensor-memory columns, repeated in
// each of the four lane quadrants.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Unswizzled shared-memory descriptor; 8-row groups of 16-byte rows are 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(128 >> 4) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// Instruction descriptor of the block-scaled e2m1 kinds, K-major operands, M = 128;
// sf_id: the first scale of the 32-bit scale cells that this instruction reads.
__device__ constexpr uint32_t idesc_fp4(int n, bool nv, uint32_t sf_id) {
    return (sf_id << 4)                          // B scale id
           | (1u << 7)                           // A format: e2m1
           | (1u << 10)                          // B format: e2m1
           | (static_cast<uint32_t>(n >> 3) << 17)
           | (nv ? 0u : (1u << 23))              // scale format: e4m3 or e8m0
           | (1u << 27)                          // M / 128
           | (sf_id << 29);                      // A scale id
}

template <bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
    if (NV)
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// The tensor scales as the two factors of a sum.  Scales on either side of 1 are one
// factor, which lies between them: a sum times 2^100 may be infinite where 2^-100 would
// bring it back.  Others stay two: their product may be infinite (2^100 each) where the sum is 0.
struct Factors {
    float a, b;
};
__device__ __forceinline__ Factors tensor_factors(const float *ga, const float *gb) {
    const float a = ga ? __ldg(ga) : 1.0f, b = gb ? __ldg(gb) : 1.0f;
    if ((a > 1.0f) != (b > 1.0f)) return Factors{__fmul_rn(a, b), 1.0f};
    return Factors{a, b};
}
__device__ __forceinline__ float scaled(float sum, const Factors &g) { return __fmul_rn(__fmul_rn(sum, g.a), g.b); }

template <int NT, bool NV, bool DEEP>
__global__ void __launch_bounds__(kThreads, DEEP ? 1 : 2)
    k_gemm_fp4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Args p) {
    using C = Cfg<NT, NV, DEEP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::STAGES * C::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // known to the compiler where there is one rank: with the join's code in it, this kernel
    // drained 128 tokens of one rank 2 us more slowly
    const int nranks = DEEP ? 1 : p.ranks, rank = DEEP ? 0 : static_cast<int>(blockIdx.x) % nranks;
    float *part = reinterpret_cast<float *>(smem);  // once all MMAs have read the stages
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->acc_full, 1);
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    pdl_wait();
    if (threadIdx.x == 0) pdl_allow_dependents();
    if (warp == 2) {
        tmem_alloc(&ctl->tmem_base, C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int *abort_flag = &ctl->abort_flag;
    const int ta = blockIdx.x / nranks;
    // this rank's stages: [kb0, kb1)
    const int nkb = (p.K + kKStage - 1) / kKStage, per = (nkb + nranks - 1) / nranks;
    const int kb0 = min(rank * per, nkb), kb1 = min(kb0 + per, nkb);
    if (warp == 0) {
        if (elect_one_sync()) {
            uint32_t armed = 0, armed_parity = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int st = (kb - kb0) % C::STAGES;
                const uint32_t ph = ((kb - kb0) / C::STAGES) & 1u;
                if (!mbar_wait_bounded(&ctl->empty[st], ph ^ 1u, abort_flag, p.err, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                uint8_t *sa = smem + st * C::STAGE, *sb = sa + kATile, *sfa = sb + C::BTILE,
                        *sfb = sfa + C::SF * kSfTile;
                const int64_t sf0 = static_cast<int64_t>(kb) * C::SF;
                const int64_t left = p.sf_tiles_k - sf0;
                const uint32_t sf_bytes = static_cast<uint32_t>(left < C::SF ? left : C::SF) * kSfTile;
                mbar_arrive_expect_tx(&ctl->full[st], kATile + C::BTILE + 2 * sf_bytes);
                armed |= 1u << st;
                armed_parity = (armed_parity & ~(1u << st)) | (ph << st);
                tma_load_2d(sa, &tmA, &ctl->full[st], kb * 128, ta * 128);
                tma_load_2d(sb, &tmB, &ctl->full[st], kb * 128, 0);
                bulk_load(sfa, p.sfa + (ta * p.sf_tiles_k + sf0) * kSfTile, sf_bytes, &ctl->full[st]);
                bulk_load(sfb, p.sfb + sf0 * kSfTile, sf_bytes, &ctl->full[st]);
            }
            if (!ok) {  // let the copies already issued land before the block exits
                for (int st = 0; st < C::STAGES; ++st)
                    if (armed & (1u << st)) {
                        const uint32_t a = smem_u32(&ctl->full[st]);
                        const uint64_t t0 = globaltimer_ns();
                        while (!mbar_try_wait(a, (armed_parity >> st) & 1u) && globaltimer_ns() - t0 < 100000000ull) {
                        }
                    }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one_sync()) {
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int st = (kb - kb0) % C::STAGES;
                const uint32_t ph = ((kb - kb0) / C::STAGES) & 1u;
                if (!mbar_wait_bounded(&ctl->full[st], ph, abort_flag, p.err, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + st * C::STAGE), sb = sa + kATile, ssfa = sb + C::BTILE,
                               ssfb = ssfa + C::SF * kSfTile;
                // A's scales, then B's, of each scale tile of the stage
                const uint32_t tsf = tmem + C::ACC + st * C::SF_COLS;
                const int kleft = p.K - kb * kKStage;
                const int nsf = kleft >= kKStage ? C::SF : (kleft + C::KSF - 1) / C::KSF;
                for (int j = 0; j < nsf; ++j) {
                    tmem_cp_scales(tsf + j * 4, smem_desc_plain(ssfa + j * kSfTile));
                    tmem_cp_scales(tsf + C::SF * 4 + j * 4, smem_desc_plain(ssfb + j * kSfTile));
                }
                const int nmma = kleft >= kKStage ? kKStage / 64 : (kleft + 63) / 64;
                for (int kk = 0; kk < nmma; ++kk) {
                    const uint64_t ad = smem_desc_sw128(sa + kk * 32, 16, 1024);
                    const uint64_t bd = smem_desc_sw128(sb + kk * 32, 16, 1024);
                    const int j = NV ? kk : kk >> 1;
                    const uint32_t id = NV ? 0u : (kk & 1) * 2u;
                    mma_fp4<NV>(tmem, ad, bd, idesc_fp4(NT, NV, id), tsf + j * 4, tsf + C::SF * 4 + j * 4,
                                (kb > kb0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(&ctl->empty[st]);
            }
            if (ok) {
                tc_commit(&ctl->acc_full);
            } else {  // wait for the MMAs already issued before tensor memory is freed
                tc_commit(&ctl->drain);
                const uint32_t a = smem_u32(&ctl->drain);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;
        const Factors g = tensor_factors(p.ga, p.gb);
        const bool ok = mbar_wait_bounded(&ctl->acc_full, 0, abort_flag, p.err, p.wait_limit_ns);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            const int row = quad * 32 + lane;
            const int64_t n = static_cast<int64_t>(ta) * 128 + row;
            const uint32_t taddr = tmem + ((quad * 32) << 16);
            if (nranks > 1) {  // a rank without stages has made no MMA: its part is 0
#pragma unroll 1
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    float v[16];
                    tmem_ld_16cols(taddr + c0, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + row] = kb1 > kb0 ? v[j] : 0.0f;
                }
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < NT; c0 += 16) {
                    float v[16];
                    tmem_ld_16cols(taddr + c0, v);
                    if (n >= p.rows_a) continue;
#pragma unroll
                    for (int j = 0; j < 16; ++j)  // a warp's 32 rows are 32 neighbours of a row of Y
                        if (c0 + j < p.rows_b)
                            p.Y[(c0 + j) * p.rows_a + n] = __float2bfloat16_rn(scaled(v[j], g));
                }
            }
        }
    }
    tc_fence_before();
    if (nranks > 1) {
        // the parts are complete in every CTA of the cluster
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const Factors g = tensor_factors(p.ga, p.gb);
        // a warp sums the 128 rows of four tokens at a time, in the order of the ranks
        const int64_t n = static_cast<int64_t>(ta) * 128 + 4 * lane;  // rows are a multiple of 8
        constexpr int kStep = kThreads / 32;
        for (int m0 = rank + nranks * warp; m0 < p.rows_b; m0 += 4 * nranks * kStep) {
            float4 sum[4] = {};
#pragma unroll 4
            for (int q = 0; q < nranks; ++q) {
                float4 x[4] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = m0 + i * nranks * kStep;
                    if (m < p.rows_b)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(x[i].x), "=f"(x[i].y), "=f"(x[i].z), "=f"(x[i].w)
                                     : "r"(map_to_rank(&part[m * 128 + 4 * lane], static_cast<uint32_t>(q))));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i].x = __fadd_rn(sum[i].x, x[i].x);
                    sum[i].y = __fadd_rn(sum[i].y, x[i].y);
                    sum[i].z = __fadd_rn(sum[i].z, x[i].z);
                    sum[i].w = __fadd_rn(sum[i].w, x[i].w);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + i * nranks * kStep;
                if (m < p.rows_b && n < p.rows_a)
                    *reinterpret_cast<uint2 *>(p.Y + m * p.rows_a + n) =
                        make_uint2(pack_bf16x2(scaled(sum[i].x, g), scaled(sum[i].y, g)),
                                   pack_bf16x2(scaled(sum[i].z, g), scaled(sum[i].w, g)));
            }
        }
        // no CTA leaves while another may read its part
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// ---------------------------------------------------------------------------- CTA pairs
// Many tokens: persistent pairs of SMs (cta_group::2).  A pair makes 256 x 256 tiles: each
// CTA stages its 128 rows of A and 128 of B's 256 (with the scales of its rows of A and of
// all of B's), the even CTA issues the MMAs, and each CTA's tensor memory holds its 128
// accumulator rows.  Per SM that reads 64 bytes of operands a clock from shared memory
// where a 128 x 256 tile of one CTA reads 96, and two thirds of its bytes from L2.
//
// Tensor memory has 512 columns: two accumulators of 256 would leave none for the scales.
// So the accumulators of consecutive tiles start at columns 0 and 96 and overlap in 160;
// the epilogue drains those first and lets the next tile's MMAs start while it drains the
// other 96.  The last 160 columns hold the scales of three stages (nv) or four (mx): before
// a stage's scales are copied, the MMAs of the stage that many before it have completed
// (its ring slot's barrier).  With two, the issuing thread's round trip through that
// barrier left the tensor pipe idle between stages (48% active; 4096 x 11008 x 4096 nv took
// 116 us).
constexpr int kPairThreads = 256;  // producer, issuer, allocator, one idle, four epilogue warps
constexpr int kAcc1 = 96;          // first column of odd tiles' accumulators
constexpr int kOverlap = 256 - kAcc1;
constexpr int kScaleBase = kAcc1 + 256;
static_assert(kOverlap % 32 == 0, "tensor memory layout");

template <bool NV>
struct PairCfg {
    static constexpr int SF = NV ? 4 : 2;
    static constexpr int KSF = NV ? 64 : 128;
    static constexpr int SF_BYTES = SF * kSfTile;  // of 128 rows
    static constexpr int STAGE = 2 * kATile + 3 * SF_BYTES;
    static constexpr int STAGES = 5;
    static constexpr int SF_COLS = SF * 12;   // scale columns of a stage: a third of A, the rest of B
    static constexpr int SF_BUFS = NV ? 3 : 4;
    static_assert(kScaleBase + SF_BUFS * SF_COLS <= 512, "tensor memory columns");
    static constexpr int OUT = 4 * 2 * 2048;  // two 32 x 32 bf16 chunks per epilogue warp
    static constexpr int SMEM = 1024 + STAGES * STAGE + OUT + 256;
    static_assert(STAGE % 1024 == 0 && SMEM <= 232448, "shared memory");
};

struct PairCtl {
    uint64_t full[5], empty[5], acc_full, acc_free, drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(PairCtl) <= 256, "control block exceeds its slot");

struct PairArgs {
    int64_t sf_tiles_k;
    int K, tiles_m, tiles;
    int64_t rows_a, rows_b;
    const float *ga, *gb;
    int *err;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool NV>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
    if (NV)
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// M = 256 in the instruction descriptor.
__device__ constexpr uint32_t idesc_fp4_pair(bool nv, uint32_t sf_id) {
    return (idesc_fp4(256, nv, sf_id) & ~(3u << 27)) | (2u << 27);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *smem_src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A stage's scale copies and MMAs (unrolled where the counts are constants).
template <bool NV>
__device__ __forceinline__ void issue_stage(uint32_t sa, uint32_t d, uint32_t tsf, int nsf, int nmma, bool accumulate) {
    using C = PairCfg<NV>;
    const uint32_t tsfb = tsf + C::SF * 4;
    const uint64_t sfa = smem_desc_plain(sa + 2 * kATile), sfb = smem_desc_plain(sa + 2 * kATile + C::SF_BYTES);
#pragma unroll
    for (int j = 0; j < C::SF; ++j)
        if (j < nsf) {  // descriptors count 16 bytes
            tmem_cp_scales_pair(tsf + j * 4, sfa + j * (kSfTile >> 4));
            tmem_cp_scales_pair(tsfb + j * 8, sfb + j * (kSfTile >> 4));
            tmem_cp_scales_pair(tsfb + j * 8 + 4, sfb + ((C::SF_BYTES + j * kSfTile) >> 4));
        }
    const uint64_t ad = smem_desc_sw128(sa, 16, 1024), bd = smem_desc_sw128(sa + kATile, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < kKStage / 64; ++kk)
        if (kk < nmma) {
            const int j = NV ? kk : kk >> 1;
            mma_fp4_pair<NV>(d, ad + 2 * kk, bd + 2 * kk, idesc_fp4_pair(NV, NV ? 0u : (kk & 1) * 2u), tsf + j * 4,
                             tsfb + j * 8, accumulate || kk > 0 ? 1u : 0u);
        }
}

template <bool NV>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    k_gemm2_fp4(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmY, const PairArgs p) {
    using C = PairCfg<NV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *out = smem + C::STAGES * C::STAGE;
    PairCtl *ctl = reinterpret_cast<PairCtl *>(out + C::OUT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->acc_full, 1);
        mbar_init(&ctl->acc_free, 8);  // four epilogue warps of each CTA
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        tma_prefetch_desc(&tmSB);
        tma_prefetch_desc(&tmY);
    }
    pdl_wait();
    if (threadIdx.x == 0) pdl_allow_dependents();
    if (warp == 2) {
        tmem_alloc_pair(&ctl->tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int *abort_flag = &ctl->abort_flag;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int nkb = (p.K + kKStage - 1) / kKStage;
    const uint32_t full0 = map_to_rank(&ctl->full[0], 0);
    const uint32_t acc_free0 = map_to_rank(&ctl->acc_free, 0);

    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer (both CTAs)
        if (elect_one_sync()) {
            uint32_t it = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            for (int t = pair; ok && t < p.tiles; t += npairs) {
                const int tm = t % p.tiles_m, tn = t / p.tiles_m;
                const int ra = tm * 2 + static_cast<int>(rank);  // 128-row tile of A
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int st = it % C::STAGES;
                    const uint32_t ph = (it / C::STAGES) & 1u;
                    if (!mbar_wait_bounded(&ctl->empty[st], ph ^ 1u, abort_flag, p.err, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + st * C::STAGE, *sb = sa + kATile, *sfa = sb + kATile, *sfb = sfa + C::SF_BYTES;
                    if (leader) {
                        mbar_arrive_expect_tx(&ctl->full[st], 2 * C::STAGE);
                        armed |= 1u << st;
                        armed_parity = (armed_parity & ~(1u << st)) | (ph << st);
                    }
                    const uint32_t bar = full0 + 8u * static_cast<uint32_t>(st);
                    tma_load_2d_pair(sa, &tmA, bar, kb * 128, ra * 128);
                    tma_load_2d_pair(sb, &tmB, bar, kb * 128, tn * 256 + static_cast<int>(rank) * 128);
                    // scale tiles are numbered along K, then along the rows; what a box takes
                    // past the end of K belongs to other rows and is not used
                    const int sf = kb * C::SF;
                    tma_load_2d_pair(sfa, &tmSA, bar, 0, static_cast<int>(ra * p.sf_tiles_k) + sf);
                    tma_load_2d_pair(sfb, &tmSB, bar, 0, static_cast<int>(2 * tn * p.sf_tiles_k) + sf);
                    tma_load_2d_pair(sfb + C::SF_BYTES, &tmSB, bar, 0, static_cast<int>((2 * tn + 1) * p.sf_tiles_k) + sf);
                }
            }
            if (!ok) {
                // Copies this CTA issued for stages the leader has not armed count on no
                // phase that can complete: give them a fixed 2 ms to land.
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) {
                }
                if (leader)
                    for (int st = 0; st < C::STAGES; ++st)
                        if (armed & (1u << st)) {
                            const uint32_t a = smem_u32(&ctl->full[st]);
                            const uint64_t t1 = globaltimer_ns();
                            while (!mbar_try_wait(a, (armed_parity >> st) & 1u) && globaltimer_ns() - t1 < 100000000ull) {
                            }
                        }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer (the leader)
        if (leader && elect_one_sync()) {
            uint32_t it = 0, local = 0;
            bool ok = true, issued = false;
            for (int t = pair; ok && t < p.tiles; t += npairs, ++local) {
                // the previous tile's overlapping columns have been drained
                if (local > 0 && !mbar_wait_bounded(&ctl->acc_free, (local - 1) & 1u, abort_flag, p.err, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + ((local & 1u) ? kAcc1 : 0);
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int st = it % C::STAGES;
                    const uint32_t ph = (it / C::STAGES) & 1u;
                    if (!mbar_wait_bounded(&ctl->full[st], ph, abort_flag, p.err, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    if (it >= C::SF_BUFS) {  // the MMAs that read this scale buffer before
                        const uint32_t o = it - C::SF_BUFS;
                        if (!mbar_wait_bounded(&ctl->empty[o % C::STAGES], (o / C::STAGES) & 1u, abort_flag, p.err,
                                               p.wait_limit_ns)) {
                            ok = false;
                            break;
                        }
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + st * C::STAGE);
                    const uint32_t tsf = tmem + kScaleBase + (it % C::SF_BUFS) * C::SF_COLS;
                    const int kleft = p.K - kb * kKStage;
                    if (kleft >= kKStage)
                        issue_stage<NV>(sa, d, tsf, C::SF, kKStage / 64, kb > 0);
                    else
                        issue_stage<NV>(sa, d, tsf, (kleft + C::KSF - 1) / C::KSF, (kleft + 63) / 64, kb > 0);
                    issued = true;
                    tc_commit_pair(&ctl->empty[st], 3);
                }
                if (ok) tc_commit_pair(&ctl->acc_full, 3);
            }
            if (!ok && issued) {  // wait for the MMAs already issued before tensor memory is freed
                tc_commit_pair(&ctl->drain, 1);
                const uint32_t a = smem_u32(&ctl->drain);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------- epilogue (both CTAs)
        const int quad = warp & 3;
        uint8_t *buf = out + quad * 4096;
        const Factors g = tensor_factors(p.ga, p.gb);
        uint32_t local = 0, chunk = 0;
        for (int t = pair; t < p.tiles; t += npairs, ++local) {
            const bool ok = mbar_wait_bounded(&ctl->acc_full, local & 1u, abort_flag, p.err, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int tm = t % p.tiles_m, tn = t / p.tiles_m;
            const int row0 = tm * 256 + static_cast<int>(rank) * 128 + quad * 32;
            const bool odd = local & 1u;
            const uint32_t taddr = tmem + ((quad * 32) << 16) + (odd ? kAcc1 : 0);
            // 32 rows of 64 bytes, 16-byte units swizzled as the output map's box.  A chunk that
            // lies outside Y takes no buffer: chunks and bulk groups are counted alike, so that
            // "all groups but the last" are those of this chunk's buffer.
            auto put = [&](const float *v, int c0) {
                if (row0 >= p.rows_a || tn * 256 + c0 >= p.rows_b) return;
                uint8_t *dst = buf + (chunk++ & 1) * 2048;
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = pack_bf16x2(scaled(v[8 * q + 2 * j], g), scaled(v[8 * q + 2 * j + 1], g));
                    *reinterpret_cast<uint4 *>(dst + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                // the map clips a chunk at the matrix's end
                if (lane == 0) tma_store_2d(&tmY, dst, tn * 256 + c0, row0);
            };
            // The columns that the next tile's accumulator overlaps go to registers first,
            // and its MMAs may start; then they are written, and the rest follows.
            const int first = odd ? 0 : kAcc1, rest = odd ? kOverlap : 0;
            float head[kOverlap / 32][32];
#pragma unroll
            for (int i = 0; i < kOverlap / 32; ++i) tmem_ld_32cols(taddr + first + 32 * i, head[i]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_free0);
#pragma unroll
            for (int i = 0; i < kOverlap / 32; ++i) put(head[i], first + 32 * i);
#pragma unroll 1
            for (int i = 0; i < kAcc1 / 32; ++i) {
                float v[32];
                tmem_ld_32cols(taddr + rest + 32 * i, v);
                put(v, rest + 32 * i);
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the pair's MMAs may still read its shared memory
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------- few tokens
// Up to 16 tokens in one launch: the weights are the rows of a tile of 128 x 16, a cluster
// of CTAs splits K, and each CTA packs its part of X into the swizzled operand tiles and
// scale tiles itself while the first weights are on their way.  The parts are joined over
// the cluster's shared memory in the order of the ranks.  The call reads the packed
// weights once; it is bound by launch and memory latency (the weights of a 4096 x 4096
// layer are 1.4 us of HBM time, the call takes 5.3), so K is split until the SMs are
// full, and a part is small enough (2048 values) for two CTAs on an SM.
constexpr int kDecTokens = 16;
constexpr int kDecThreads = 256;    // producer, issuer (after packing), packers, of which four drain
constexpr int kDecMaxSlice = 2048;  // K values of a CTA
constexpr int kDecStages = 4;
constexpr int kDecTmem = 256;       // two CTAs share an SM's 512 columns
constexpr int kDecSms = 148;        // of a B200; the workspace's size, which follows, is asked for without a device

template <bool NV>
struct DecCfg {
    static constexpr int SF = NV ? 4 : 2;
    static constexpr int KSF = NV ? 64 : 128;
    static constexpr int STAGE = kATile + 2048;  // A and its scale tiles (mx uses half of that)
    static constexpr int XTILE = kDecTokens * 128;
    static constexpr int XSTAGES = kDecMaxSlice / kKStage;
    static constexpr int SMEM = 1024 + kDecStages * STAGE + XSTAGES * (XTILE + SF * kSfTile) + 256;
    static constexpr int SF_COLS = SF * 8;
    static constexpr int RED = 128 * (kDecTokens + 1) * 4;  // the parts, in the stages' place
    static_assert(32 + kDecStages * SF_COLS <= kDecTmem && SMEM <= 113 * 1024 && RED <= kDecStages * STAGE,
                  "two blocks per SM");
};

// Doubles the ranks that split K while every SM has one CTA at most and every rank `least`
// stages, or (`two`) two CTAs of at least eight stages.  On 11008 x 4096 (86 tiles) two ranks
// take 7.9 us for one token where one takes 9.9.
int split_ranks(int64_t tiles, int64_t stages, int ranks, int sms, int least, bool two) {
    while (ranks < 8 && ((2 * ranks * tiles <= sms && stages >= 2 * least * ranks) ||
                         (two && 2 * ranks * tiles <= 2 * sms && stages >= 16 * ranks)))
        ranks *= 2;
    return ranks;
}

// Enough ranks for the slice that a CTA can pack, at least.
int decode_ranks(int64_t N, int64_t K) {
    int ranks = 1;
    while (static_cast<int64_t>(ranks) * kDecMaxSlice < K && ranks < 16) ranks *= 2;
    return split_ranks((N + 127) / 128, (K + kKStage - 1) / kKStage, ranks, kDecSms, 2, true);
}
int64_t decode_slice(int64_t N, int64_t K) {
    const int64_t stages = (K + kKStage - 1) / kKStage, ranks = decode_ranks(N, K);
    return (stages + ranks - 1) / ranks * kKStage;
}

struct DecArgs {
    const __nv_bfloat16 *X;
    const uint8_t *sf;
    const float *gx, *gw;
    __nv_bfloat16 *Y;
    int64_t sf_tiles_k, N, K;
    int M, slice;  // K values per rank, a multiple of kKStage
    int ranks;     // CTAs of a cluster
    int *err;
    uint64_t wait_limit_ns;
};

struct DecCtl {
    uint64_t full[kDecStages], empty[kDecStages], acc_full, drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(DecCtl) <= 256, "control block exceeds its slot");

// Packs the CTA's slice of X: token r, values k0 .. k0 + 15 of the slice per step.
template <bool NV>
__device__ __forceinline__ void pack_slice(const DecArgs &p, int64_t kbase, int klen, uint8_t *xt, uint8_t *xs, int first,
                                           int count) {
    using C = DecCfg<NV>;
    const float g = NV && p.gx ? __ldg(p.gx) : 1.0f, inv_g = __fdiv_rn(1.0f, g);
    const int per_row = (klen + 63) / 64 * 4;  // the last MMA's values past K are packed as 0
    const int total = p.M * per_row;
    for (int i0 = first - (first & 31); i0 < total; i0 += count) {
        const int i = i0 + (first & 31);
        const int r = i / per_row, k = (i - r * per_row) * 16;
        const bool live = i < total, in = live && k < klen;
        float x[16];
        if (in) {
            fp4::load16<__nv_bfloat16>(p.X + static_cast<int64_t>(r) * p.K + kbase + k, x);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        }
        const fp4::Coded c = fp4::encode<NV>(x, g, inv_g);
        if (!live) continue;
        const int st = k / kKStage, byte = (k % kKStage) / 2;
        *reinterpret_cast<uint2 *>(xt + st * C::XTILE + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 8)) =
            make_uint2(c.lo, c.hi);
        const int block = k / (NV ? 16 : 32);
        if (NV || (k & 16) == 0) xs[(block / 4) * kSfTile + r * 16 + (block & 3)] = in ? c.scale : 0;
    }
}

template <bool NV>
__global__ void __launch_bounds__(kDecThreads, 2) k_decode_fp4(const __grid_constant__ CUtensorMap tmW, const DecArgs p) {
    using C = DecCfg<NV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *xt = smem + kDecStages * C::STAGE, *xs = xt + C::XSTAGES * C::XTILE;
    DecCtl *ctl = reinterpret_cast<DecCtl *>(xs + C::XSTAGES * C::SF * kSfTile);
    float *red = reinterpret_cast<float *>(smem);  // once all MMAs have read the stages
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t nranks = static_cast<uint32_t>(p.ranks), rank = blockIdx.x % nranks;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDecStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->acc_full, 1);
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmW);
    }
    pdl_wait();
    if (threadIdx.x == 0) pdl_allow_dependents();
    if (warp == 2) {
        tmem_alloc(&ctl->tmem_base, kDecTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int *abort_flag = &ctl->abort_flag;
    const int tile = blockIdx.x / nranks;
    const int64_t kbase = static_cast<int64_t>(rank) * p.slice;
    const int klen = static_cast<int>(p.K - kbase < p.slice ? (p.K > kbase ? p.K - kbase : 0) : p.slice);
    const int nkb = (klen + kKStage - 1) / kKStage;
    bool ok = true;

    if (warp == 0) {
        if (elect_one_sync()) {
            uint32_t armed = 0, armed_parity = 0;
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % kDecStages;
                const uint32_t ph = (kb / kDecStages) & 1u;
                if (!mbar_wait_bounded(&ctl->empty[st], ph ^ 1u, abort_flag, p.err, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                uint8_t *sa = smem + st * C::STAGE;
                const int64_t sf0 = kbase / C::KSF + static_cast<int64_t>(kb) * C::SF;
                const int64_t left = p.sf_tiles_k - sf0;
                const uint32_t sf_bytes = static_cast<uint32_t>(left < C::SF ? left : C::SF) * kSfTile;
                mbar_arrive_expect_tx(&ctl->full[st], kATile + sf_bytes);
                armed |= 1u << st;
                armed_parity = (armed_parity & ~(1u << st)) | (ph << st);
                tma_load_2d(sa, &tmW, &ctl->full[st], static_cast<int>(kbase / 2) + kb * 128, tile * 128);
                bulk_load(sa + kATile, p.sf + (tile * p.sf_tiles_k + sf0) * kSfTile, sf_bytes, &ctl->full[st]);
            }
            if (!ok) {  // let the copies already issued land before the block exits
                for (int st = 0; st < kDecStages; ++st)
                    if (armed & (1u << st)) {
                        const uint32_t a = smem_u32(&ctl->full[st]);
                        const uint64_t t0 = globaltimer_ns();
                        while (!mbar_try_wait(a, (armed_parity >> st) & 1u) && globaltimer_ns() - t0 < 100000000ull) {
                        }
                    }
            }
        }
        __syncwarp();
    } else {
        pack_slice<NV>(p, kbase, klen, xt, xs, static_cast<int>(threadIdx.x) - 32, kDecThreads - 32);
        fence_proxy_async_smem();
        asm volatile("bar.sync 1, %0;" ::"n"(kDecThreads - 32) : "memory");
    }
    if (warp == 1) {
        if (elect_one_sync()) {
            for (int kb = 0; kb < nkb; ++kb) {
                const int st = kb % kDecStages;
                const uint32_t ph = (kb / kDecStages) & 1u;
                if (!mbar_wait_bounded(&ctl->full[st], ph, abort_flag, p.err, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + st * C::STAGE), ssfa = sa + kATile;
                const uint32_t sb = smem_u32(xt + kb * C::XTILE), ssfb = smem_u32(xs + kb * C::SF * kSfTile);
                const uint32_t tsf = tmem + 32 + st * C::SF_COLS;
                const int kleft = klen - kb * kKStage;
                const int nsf = kleft >= kKStage ? C::SF : (kleft + C::KSF - 1) / C::KSF;
                for (int j = 0; j < nsf; ++j) {
                    tmem_cp_scales(tsf + j * 4, smem_desc_plain(ssfa + j * kSfTile));
                    tmem_cp_scales(tsf + C::SF * 4 + j * 4, smem_desc_plain(ssfb + j * kSfTile));
                }
                const int nmma = kleft >= kKStage ? kKStage / 64 : (kleft + 63) / 64;
                for (int kk = 0; kk < nmma; ++kk) {
                    const int j = NV ? kk : kk >> 1;
                    mma_fp4<NV>(tmem, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sb + kk * 32, 16, 1024),
                                idesc_fp4(kDecTokens, NV, NV ? 0u : (kk & 1) * 2u), tsf + j * 4, tsf + C::SF * 4 + j * 4,
                                (kb > 0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(&ctl->empty[st]);
            }
            if (ok) {
                tc_commit(&ctl->acc_full);
            } else {  // wait for the MMAs already issued before tensor memory is freed
                tc_commit(&ctl->drain);
                const uint32_t a = smem_u32(&ctl->drain);
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < 100000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const bool done = mbar_wait_bounded(&ctl->acc_full, 0, abort_flag, p.err, p.wait_limit_ns);
        if (__all_sync(0xffffffffu, done)) {
            tc_fence_after();
            const int row = (warp & 3) * 32 + lane;
            float v[16];
            tmem_ld_16cols(tmem + (((warp & 3) * 32) << 16), v);
            // a rank without a part of K has made no MMA: its part is 0
#pragma unroll
            for (int j = 0; j < kDecTokens; ++j) red[row * (kDecTokens + 1) + j] = nkb > 0 ? v[j] : 0.0f;
        }
    }
    tc_fence_before();
    // the parts are complete in every CTA of the cluster
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const Factors g = tensor_factors(p.gx, p.gw);
    const int rows = 128 / static_cast<int>(nranks);  // of this rank
    for (int i = threadIdx.x; i < rows * p.M; i += kDecThreads) {
        const int row = static_cast<int>(rank) * rows + i % rows, m = i / rows;
        const int64_t n = static_cast<int64_t>(tile) * 128 + row;
        float sum = 0.0f;
        for (uint32_t q = 0; q < nranks; ++q) {
            float part;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(part)
                         : "r"(map_to_rank(&red[row * (kDecTokens + 1) + m], q)));
            sum = __fadd_rn(sum, part);
        }
        if (n < p.N) p.Y[static_cast<int64_t>(m) * p.N + n] = __float2bfloat16_rn(scaled(sum, g));
    }
    // no CTA leaves while another may read its part
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kDecTmem);
    }
}

cudaLaunchAttribute cluster_of(int ranks) {
    cudaLaunchAttribute cluster{};
    cluster.id = ranks > 1 ? cudaLaunchAttributeClusterDimension : cudaLaunchAttributeIgnore;
    cluster.val.clusterDim.x = static_cast<unsigned>(ranks);
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    return cluster;
}

struct Side {
    const uint8_t *codes, *scales;
    const float *g;
    int64_t rows;
};

template <int NT, bool NV, bool DEEP>
cudaError_t launch_t(const Side &a, const Side &b, int64_t K, int ranks, void *Y, const DeviceInfo &dev,
                     cudaStream_t st) {
    using C = Cfg<NT, NV, DEEP>;
    CUtensorMap ma, mb;
    cudaError_t e = encode_map_2d(ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, K / 2, a.rows, K / 2, 128, 128,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    e = encode_map_2d(mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b.codes, K / 2, b.rows, K / 2, 128, NT,
                      CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    auto kern = k_gemm_fp4<NT, NV, DEEP>;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev.device & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    Args p{};
    p.sfa = a.scales;
    p.sfb = b.scales;
    p.sf_tiles_k = (K / (NV ? 16 : 32) + 3) / 4;
    p.rows_a = a.rows;
    p.rows_b = b.rows;
    p.ranks = ranks;
    p.K = static_cast<int>(K);
    p.ga = a.g;
    p.gb = b.g;
    p.Y = static_cast<__nv_bfloat16 *>(Y);
    p.err = device_error_word();
    if (!p.err) return cudaErrorInvalidSymbol;
    p.wait_limit_ns = kWaitLimitNs;
    const int64_t tiles = (a.rows + 127) / 128;  // rows are below 2^31
    return launch_pdl_ex(kern, dim3(static_cast<unsigned>(tiles * ranks)), dim3(kThreads), C::SMEM, st,
                         cluster_of(ranks), ma, mb, p);
}

template <bool NV>
cudaError_t launch_pair(const Side &a, const Side &b, int64_t K, void *Y, const DeviceInfo &dev, cudaStream_t st) {
    using C = PairCfg<NV>;
    const int64_t tiles_k = (K / (NV ? 16 : 32) + 3) / 4;
    CUtensorMap ma, mb, sa, sb, my;
    auto codes = [&](CUtensorMap &m, const Side &s) {
        return encode_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, s.codes, K / 2, s.rows, K / 2, 128, 128,
                             CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto scales = [&](CUtensorMap &m, const Side &s) {  // one scale tile per row of the map
        return encode_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, s.scales, kSfTile / 4, (s.rows + 127) / 128 * tiles_k,
                             kSfTile, kSfTile / 4, C::SF, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    cudaError_t e;
    if ((e = codes(ma, a)) != cudaSuccess || (e = codes(mb, b)) != cudaSuccess || (e = scales(sa, a)) != cudaSuccess ||
        (e = scales(sb, b)) != cudaSuccess ||
        (e = encode_map_2d(my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, b.rows, a.rows, b.rows * 2, 32, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B)) != cudaSuccess)
        return e;
    auto kern = k_gemm2_fp4<NV>;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev.device & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    PairArgs p{};
    p.sf_tiles_k = tiles_k;
    p.K = static_cast<int>(K);
    p.tiles_m = static_cast<int>((a.rows + 255) / 256);
    const int64_t tiles = p.tiles_m * ((b.rows + 255) / 256);
    // scale tiles are numbered in 32 bits
    if (tiles > 0x7FFFFFFF || ((std::max(a.rows, b.rows) + 255) / 256 * 2 + 1) * tiles_k > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    p.tiles = static_cast<int>(tiles);
    p.rows_a = a.rows;
    p.rows_b = b.rows;
    p.ga = a.g;
    p.gb = b.g;
    p.err = device_error_word();
    if (!p.err) return cudaErrorInvalidSymbol;
    p.wait_limit_ns = kWaitLimitNs;
    const int grid = 2 * static_cast<int>(std::min<int64_t>(tiles, dev.sm_count / 2));
    return launch_pdl(kern, dim3(grid), dim3(kPairThreads), C::SMEM, st, ma, mb, sa, sb, my, p);
}

// Up to 128 tokens: from eight stages on, K is split over the ranks of a cluster (64 tokens
// of 4096 x 4096 take 9.2 us where one rank takes 11.5; on 1024 x 1024, four stages, two ranks
// take 7.4 where one takes 6.8).  The join of 128 columns costs more: such ranks have four
// stages, and do not share an SM.  One rank has the deep ring if it has its SM for itself (its
// three stages took 2 us more for 128 tokens of 1024 x 1024); clusters do not, since an SM may then hold two of their CTAs (16 clusters of 8 do not find
// 8 free SMs in a group each: 17 tokens of 2048 x 8192 13.4 us against 9.3).
template <int NT, bool NV>
cudaError_t launch_few(const Side &w, const Side &x, int64_t K, void *Y, const DeviceInfo &dev, cudaStream_t st) {
    const int64_t tiles = (w.rows + 127) / 128, stages = (K + kKStage - 1) / kKStage;
    const int ranks = stages < 8 ? 1 : split_ranks(tiles, stages, 1, dev.sm_count, NT <= 64 ? 2 : 4, NT <= 64);
    return ranks == 1 && tiles <= dev.sm_count ? launch_t<NT, NV, true>(w, x, K, ranks, Y, dev, st)
                                               : launch_t<NT, NV, false>(w, x, K, ranks, Y, dev, st);
}

template <bool NV>
cudaError_t dispatch(const Side &x, const Side &w, int64_t K, void *Y, const DeviceInfo &dev, cudaStream_t st) {
    const int64_t M = x.rows;
    if (M <= 16) return launch_few<16, NV>(w, x, K, Y, dev, st);
    if (M <= 32) return launch_few<32, NV>(w, x, K, Y, dev, st);
    if (M <= 64) return launch_few<64, NV>(w, x, K, Y, dev, st);
    if (M <= 128) return launch_few<128, NV>(w, x, K, Y, dev, st);
    return launch_pair<NV>(x, w, K, Y, dev, st);
}

template <bool NV>
cudaError_t launch_decode(const void *X, const float *gx, const Side &w, int64_t M, int64_t K, void *Y,
                          const DeviceInfo &dev, cudaStream_t st) {
    using C = DecCfg<NV>;
    CUtensorMap map;
    cudaError_t e = encode_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, K / 2, w.rows, K / 2, 128, 128,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    auto kern = k_decode_fp4<NV>;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev.device & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    const int64_t tiles = (w.rows + 127) / 128;
    const int ranks = decode_ranks(w.rows, K);
    if (ranks > 8 || tiles * ranks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    DecArgs p{};
    p.X = static_cast<const __nv_bfloat16 *>(X);
    p.sf = w.scales;
    p.gx = gx;
    p.gw = w.g;
    p.Y = static_cast<__nv_bfloat16 *>(Y);
    p.sf_tiles_k = (K / (NV ? 16 : 32) + 3) / 4;
    p.N = w.rows;
    p.K = K;
    p.M = static_cast<int>(M);
    p.ranks = ranks;
    p.slice = static_cast<int>(decode_slice(w.rows, K));
    p.err = device_error_word();
    if (!p.err) return cudaErrorInvalidSymbol;
    p.wait_limit_ns = kWaitLimitNs;
    return launch_pdl_ex(kern, dim3(static_cast<unsigned>(tiles * ranks)), dim3(kDecThreads), C::SMEM, st,
                         cluster_of(ranks), map, p);
}

}  // namespace

// The product packs X itself while that is little work for a CTA, 8 tokens by 1024 values
// or 4 by 2048, and no second wave of CTAs does it again.  At the border both ways take
// the same (8 tokens on 4096 x 4096 7.7 us, 9 packed apart 8.0); 1 token on 28672 x 8192, 896
// CTAs, took 32.0 us where packing apart takes 27.
bool fp4_packs_in_product(int64_t M, int64_t N, int64_t K) {
    return M <= kDecTokens && K <= 8ll * kDecMaxSlice && M * decode_slice(N, K) <= 8 * 1024 &&
           (N + 127) / 128 * decode_ranks(N, K) <= 2 * kDecSms;
}

cudaError_t launch_fp4_few_tokens(const void *X, const float *gx, const uint8_t *w_codes, const uint8_t *w_scales,
                                  const float *gw, bool nv, int64_t M, int64_t N, int64_t K, void *Y,
                                  const DeviceInfo &dev, cudaStream_t st) {
    const Side w{w_codes, w_scales, gw, N};
    return nv ? launch_decode<true>(X, gx, w, M, K, Y, dev, st) : launch_decode<false>(X, gx, w, M, K, Y, dev, st);
}

cudaError_t launch_gemm_fp4(const uint8_t *x_codes, const uint8_t *x_scales, const float *gx, const uint8_t *w_codes,
                            const uint8_t *w_scales, const float *gw, bool nv, int64_t M, int64_t N, int64_t K,
                            void *Y, const DeviceInfo &dev, cudaStream_t st) {
    const Side x{x_codes, x_scales, gx, M}, w{w_codes, w_scales, gw, N};
    return nv ? dispatch<true>(x, w, K, Y, dev, st) : dispatch<false>(x, w, K, Y, dev, st);
}

}  // namespace eqat
