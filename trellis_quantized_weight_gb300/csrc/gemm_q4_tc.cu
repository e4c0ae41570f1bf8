// Products with 4-bit weights for many activation rows, on the 5th-generation tensor cores.
//
//   D[n, m] (tensor memory, fp32) = sum over a group's k of (c[n, k] - 8) x[m, k]     128 weight rows, NB activation rows
//   o[n, m] (registers, fp32)    += scale[n, g] D[n, m] + (bias + 8 scale)[n, g] sum_k x[m, k]
//
// The codes minus 8 and the activations are exact in bf16, so no weight is rounded; a group's sum leaves the
// accumulators after its own products and is scaled in fp32.  That costs a read of tensor memory and a multiply-add for
// each output and group, by warps that have nothing else to do: it stays behind the tensor cores as long as a group is
// long enough.
//
// A CTA has 20 warps: one loads code tiles, one activation tiles, one issues the products, one keeps tensor
// memory, 8 turn codes into bf16 pairs in tensor memory (the products' first operand), 8 take the
// groups' sums.  Tiles are 128 rows x NB; a CTA takes tile after tile (those of one weight row block next to
// each other, so that codes come from L2), and where there are few tiles a cluster of CTAs shares the k of
// one and adds its parts in shared memory in their order.
//
// The sums of x over each group, for weights with biases, and activations in 8 bits as bf16, are made by a
// small kernel before.
#include <cuda.h>
#include <cooperative_groups.h>
#include <mutex>

#include "gemm_q4.cuh"

namespace trellis {

__device__ unsigned int g_q4_error = 0u;

namespace {

namespace cg = cooperative_groups;

constexpr int kTcRows = 128;                 // weight rows of a tile
constexpr int kTcStageK = 128;               // k of a stage
constexpr int kCodeBytes = kTcRows * 128;    // a code tile: 256 k (two stages) of 128 rows
constexpr int kDecodeWarps = 8, kSumWarps = 8;
constexpr int kTcThreads = 32 * (4 + kDecodeWarps + kSumWarps);

// Slots: D buffers of NB columns and A slots of 64 columns fill the 512 of tensor memory.
template <int G, int NB>
struct TcShape {
    static constexpr int kPer = kTcStageK / G;                      // groups of a stage
    static constexpr int kD = NB == 32 ? 8 : NB == 64 ? 4 : 2;
    static constexpr int kA = (512 - kD * NB) / 64 < 4 ? (512 - kD * NB) / 64 : 4;
    static constexpr int kXTile = NB * kTcStageK * 2;               // two boxes of 64 k
    static constexpr int kXBytes = kXTile + (kPer * NB * 4 + 1023) / 1024 * 1024;      // and the sums of its groups
    static constexpr int kX = NB == 192 ? 3 : NB == 128 ? 4 : NB == 64 ? 6 : 8;
    static constexpr int kCode = NB >= 128 ? 2 : 5;
    static constexpr int kOffX = 0, kOffCode = kX * kXBytes, kOffBar = kOffCode + kCode * kCodeBytes;
    static constexpr int kBarX = 0, kBarXEmpty = kX, kBarCode = 2 * kX, kBarCodeEmpty = 2 * kX + kCode;
    static constexpr int kBarA = 2 * (kX + kCode), kBarAEmpty = kBarA + kA, kBarD = kBarA + 2 * kA, kBarDEmpty = kBarD + kD;
    static constexpr int kBarSums = kBarDEmpty + kD, kBars = kBarSums + 1;
    static constexpr int kOffTaddr = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffTaddr + 16 + 1024;             // the base is rounded up to 1 KB
    static constexpr uint32_t kInstr = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NB >> 3) << 17) |
                                       (static_cast<uint32_t>(kTcRows >> 4) << 24);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    static_assert(kD * NB + kA * 64 <= 512 && kA >= 2, "tensor memory");
    static_assert(kTcRows * NB * 4 <= kX * kXBytes, "a part of the sums fits where activations were");
};

struct TcArgs {
    const uint16_t *scales, *biases;
    const float *x_scales, *sums;       // sums [groups, m_pad]
    uint16_t* out;
    int M, K, N, groups, m_pad;
    int m_tiles, tiles, parts;
};

// ---- waits --------------------------------------------------------------------------
// Every wait is bounded, as the other tensor-core kernels' are: one that runs out sets the error word and its
// warp leaves its loops; copies in flight are waited for, tensor memory is given back.
constexpr unsigned long long kWaitNs = 2000000000ull;   // 2 s
constexpr uint32_t kWaitPollCap = 1u << 26;

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0u;
}
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t i = 0; i < kWaitPollCap; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 63u) == 63u) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (t - t0 > kWaitNs) break;
        }
    }
    atomicOr(&g_q4_error, 1u);
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    return mbar_try(bar, parity) || mbar_wait_long(bar, parity);
}

// A place in a ring of kSlots and the parity of its turn.
template <int kSlots>
struct Ring {
    int slot = 0;
    uint32_t turn = 0u;
    __device__ __forceinline__ void next() {
        if (++slot == kSlots) { slot = 0; turn ^= 1u; }
    }
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// K-major, 128-byte swizzle: 1 KB between atoms of 8 rows, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, uint32_t accumulate) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(instr), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
// The registers are operands, so that nothing takes them before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// Codes 2i and 2i + 1 of a word as a bf16 pair of c - 8, i = 0 .. 3: a byte goes to both halves, the upper one's from
// the word shifted by a code.
__device__ __forceinline__ void pairs_in_order(uint32_t w, uint32_t* p) {
    const uint32_t u = w >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t both = __byte_perm(w, u, static_cast<uint32_t>(i) | (static_cast<uint32_t>(i) << 4) |
                                                    (static_cast<uint32_t>(4 + i) << 8) | (static_cast<uint32_t>(4 + i) << 12));
        const uint32_t c = (both & 0x000f000fu) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(c), "r"(0x43084308u));
    }
}

template <int G, int NB, bool kBias>
__global__ void __launch_bounds__(kTcThreads, 1)
q4_tc_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap code_map, const __grid_constant__ CUtensorMap x_map) {
    using S = TcShape<G, NB>;
    constexpr int kPer = S::kPer, kCols = NB / 2;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    unsigned char* const smem = smem_raw + (sbase - sraw);
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kX; ++i) {
            mbar_init(bar(S::kBarX + i), 1);
            mbar_init(bar(S::kBarXEmpty + i), 1 + (kBias ? kSumWarps : 0));
        }
        for (int i = 0; i < S::kCode; ++i) {
            mbar_init(bar(S::kBarCode + i), 1);
            mbar_init(bar(S::kBarCodeEmpty + i), kDecodeWarps);
        }
        for (int i = 0; i < S::kA; ++i) {
            mbar_init(bar(S::kBarA + i), kDecodeWarps);
            mbar_init(bar(S::kBarAEmpty + i), 1);
        }
        for (int i = 0; i < S::kD; ++i) {
            mbar_init(bar(S::kBarD + i), 1);
            mbar_init(bar(S::kBarDEmpty + i), kSumWarps);
        }
        mbar_init(bar(S::kBarSums), kSumWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(sbase + S::kOffTaddr), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t taddr = *reinterpret_cast<volatile uint32_t*>(smem + S::kOffTaddr);
    const uint32_t t_a = taddr + S::kD * NB;

    // this CTA's share of k, in blocks of two stages, and its first tile
    const int part = a.parts > 1 ? static_cast<int>(blockIdx.x) % a.parts : 0;
    const int blocks = (a.K + 2 * kTcStageK - 1) / (2 * kTcStageK), stages = (a.K + kTcStageK - 1) / kTcStageK;
    const int b0 = static_cast<int>(static_cast<long long>(blocks) * part / a.parts);
    const int b1 = static_cast<int>(static_cast<long long>(blocks) * (part + 1) / a.parts);
    const int s0 = 2 * b0, s1 = min(2 * b1, stages);
    const int tile0 = a.parts > 1 ? static_cast<int>(blockIdx.x) / a.parts : static_cast<int>(blockIdx.x);
    const int tile_step = a.parts > 1 ? a.tiles : static_cast<int>(gridDim.x);
    if (warp == 0 && lane == 0) {
        // L2 prefetches only: nothing reaches the CTA before the wait for the previous grid
        for (int b = b0; b < b1 && b < b0 + S::kCode; ++b)
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                         :: "l"(reinterpret_cast<uint64_t>(&code_map)), "r"(b * 32), "r"(tile0 / a.m_tiles * kTcRows) : "memory");
    }
    griddep_wait();

    bool alive = true;
    if (warp < 4) {
        if constexpr (NB >= 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------------ code tiles
            Ring<S::kCode> r;
            int issued = 0;
            for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
                const int n0 = tile / a.m_tiles * kTcRows;
                for (int b = b0; b < b1; ++b) {
                    alive = mbar_wait(bar(S::kBarCodeEmpty + r.slot), r.turn ^ 1u);
                    if (!alive) break;
                    mbar_expect(bar(S::kBarCode + r.slot), kCodeBytes);
                    tma_load_2d(sbase + S::kOffCode + r.slot * kCodeBytes, &code_map, b * 32, n0, bar(S::kBarCode + r.slot));
                    r.next();
                    ++issued;
                }
            }
            // what was asked for has landed before the CTA ends
            for (int i = max(issued - S::kCode, 0); i < issued; ++i) (void)mbar_wait(bar(S::kBarCode + i % S::kCode), (i / S::kCode) & 1);
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------------------ activation tiles
            Ring<S::kX> r;
            int issued = 0;
            for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
                const int m0 = tile % a.m_tiles * NB;
                for (int s = s0; s < s1; ++s) {
                    alive = mbar_wait(bar(S::kBarXEmpty + r.slot), r.turn ^ 1u);
                    if (!alive) break;
                    const uint32_t full = bar(S::kBarX + r.slot), dst = sbase + S::kOffX + r.slot * S::kXBytes;
                    const int sums = kBias ? min(kPer, a.groups - s * kPer) : 0;
                    mbar_expect(full, static_cast<uint32_t>(S::kXTile + sums * NB * 4));
                    tma_load_2d(dst, &x_map, s * kTcStageK, m0, full);
                    tma_load_2d(dst + NB * 128, &x_map, s * kTcStageK + 64, m0, full);
                    for (int q = 0; q < sums; ++q)
                        bulk_load(dst + S::kXTile + q * NB * 4, a.sums + static_cast<size_t>(s * kPer + q) * a.m_pad + m0, NB * 4, full);
                    r.next();
                    ++issued;
                }
            }
            for (int i = max(issued - S::kX, 0); i < issued; ++i) (void)mbar_wait(bar(S::kBarX + i % S::kX), (i / S::kX) & 1);
        } else if (warp == 2 && lane == 0) {
            // ------------------------------------------------------------ products
            Ring<S::kX> x;
            Ring<S::kA> c;
            Ring<S::kD> d;
            const uint64_t desc0 = smem_desc(sbase + S::kOffX);
            const uint32_t desc_hi = static_cast<uint32_t>(desc0 >> 32);
            int last = -1;
            uint32_t last_turn = 0u;
            for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
                for (int s = s0; s < s1 && alive; ++s) {
                    alive = mbar_wait(bar(S::kBarX + x.slot), x.turn) && mbar_wait(bar(S::kBarA + c.slot), c.turn);
                    if (!alive) break;
                    fence_after();
                    const uint32_t desc = static_cast<uint32_t>(desc0) + static_cast<uint32_t>(x.slot * (S::kXBytes >> 4));
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        if (s * kPer + q >= a.groups) break;
                        alive = mbar_wait(bar(S::kBarDEmpty + d.slot), d.turn ^ 1u);
                        if (!alive) break;
                        fence_after();
#pragma unroll
                        for (int kk = 0; kk < G / 16; ++kk) {
                            const int k = q * (G / 16) + kk;                      // step of 16 in the stage
                            const uint32_t lo = desc + static_cast<uint32_t>(((k >> 2) * (NB * 128) + (k & 3) * 32) >> 4);
                            mma_ta(taddr + d.slot * NB, t_a + c.slot * 64 + 8 * k, (static_cast<uint64_t>(desc_hi) << 32) | lo, S::kInstr,
                                   kk > 0 ? 1u : 0u);
                        }
                        mma_commit(bar(S::kBarD + d.slot));
                        last = d.slot;
                        last_turn = d.turn;
                        d.next();
                    }
                    if (!alive) break;
                    mma_commit(bar(S::kBarAEmpty + c.slot));
                    mma_commit(bar(S::kBarXEmpty + x.slot));
                    x.next();
                    c.next();
                }
            }
            // the last products are done before tensor memory is given back
            if (last >= 0) (void)mbar_wait(bar(S::kBarD + last), last_turn);
        }
        __syncwarp();
    } else if (warp < 4 + kDecodeWarps) {
        if constexpr (NB >= 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // ---------------------------------------------------------------- codes to bf16
        const int quarter = warp & 3, half = (warp - 4) >> 2;           // 32 rows; 64 k of each stage
        const int row = 32 * quarter + lane;
        const uint32_t t_row = t_a + (static_cast<uint32_t>(32 * quarter) << 16) + 32 * half;
        const uint32_t row_at = sbase + S::kOffCode + row * 128, r7 = row & 7;
        Ring<S::kCode> r;
        Ring<S::kA> c;
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
            for (int s = s0; s < s1; ++s) {
                if ((s & 1) == 0) alive = mbar_wait(bar(S::kBarCode + r.slot), r.turn);
                if (!alive) break;
                const uint32_t at = row_at + r.slot * kCodeBytes;
                const uint32_t chunk = 4 * (s & 1) + 2 * half;
                const uint4 lo = lds128(at + ((chunk ^ r7) << 4)), hi = lds128(at + (((chunk + 1) ^ r7) << 4));
                uint32_t p[16], u[16];
                pairs_in_order(lo.x, p); pairs_in_order(lo.y, p + 4); pairs_in_order(lo.z, p + 8); pairs_in_order(lo.w, p + 12);
                pairs_in_order(hi.x, u); pairs_in_order(hi.y, u + 4); pairs_in_order(hi.z, u + 8); pairs_in_order(hi.w, u + 12);
                if ((s & 1) == 1 || s + 1 == s1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::kBarCodeEmpty + r.slot));
                    r.next();
                }
                alive = mbar_wait(bar(S::kBarAEmpty + c.slot), c.turn ^ 1u);
                if (!alive) break;
                fence_after();
                tmem_st16(t_row + c.slot * 64, p);
                tmem_st16(t_row + c.slot * 64 + 16, u);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::kBarA + c.slot));
                c.next();
            }
        }
    } else {
        if constexpr (NB >= 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        // ---------------------------------------------------------------- sums of the groups
        const int quarter = warp & 3, half = (warp - 4 - kDecodeWarps) >> 2;
        const uint32_t t_row = taddr + (static_cast<uint32_t>(32 * quarter) << 16) + kCols * half;
        Ring<S::kX> x;
        Ring<S::kD> d;
        float2 o[kCols / 2];
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
            const int m0 = tile % a.m_tiles * NB + kCols * half;
            const int n = tile / a.m_tiles * kTcRows + 32 * quarter + lane;
            const size_t row = static_cast<size_t>(min(n, a.N - 1)) * a.groups;
            const uint16_t* scales = a.scales + row;
            const uint16_t* biases = kBias ? a.biases + row : nullptr;
            const int g0 = s0 * kPer, g1 = min(s1 * kPer, a.groups);
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) o[j] = make_float2(0.0f, 0.0f);
            uint32_t s_next = g0 < g1 ? __ldg(scales + g0) : 0u, b_next = kBias && g0 < g1 ? __ldg(biases + g0) : 0u;
            for (int g = g0; g < g1; ++g) {
                const float scale = __uint_as_float(s_next << 16);
                const float bias = kBias ? fmaf(8.0f, scale, __uint_as_float(b_next << 16)) : 0.0f;
                if (g + 1 < g1) {
                    s_next = __ldg(scales + g + 1);
                    if constexpr (kBias) b_next = __ldg(biases + g + 1);
                }
                const int q = g % kPer;
                alive = mbar_wait(bar(S::kBarD + d.slot), d.turn);
                if (alive && kBias && q == 0) alive = mbar_wait(bar(S::kBarX + x.slot), x.turn);
                if (!alive) break;
                fence_after();
                const float4* sums = reinterpret_cast<const float4*>(smem + S::kOffX + x.slot * S::kXBytes + S::kXTile + q * NB * 4) + kCols / 4 * half;
                constexpr int kBufs = NB == 192 ? 1 : 2;         // 192: there are no registers for a second one
                uint32_t v[kBufs][16];
                if (kBufs == 2) tmem_ld16(v[0], t_row + d.slot * NB);
#pragma unroll
                for (int i = 0; i < kCols / 16; ++i) {
                    uint32_t(&now)[16] = v[i % kBufs];
                    if (kBufs == 1) tmem_ld16(now, t_row + d.slot * NB + 16 * i);
                    tmem_wait_ld(now);
                    if (i + 1 < kCols / 16) {
                        if (kBufs == 2) tmem_ld16(v[(i + 1) % kBufs], t_row + d.slot * NB + 16 * (i + 1));
                    } else {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(S::kBarDEmpty + d.slot));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float2& y = o[8 * i + j];
                        y = __ffma2_rn(make_float2(scale, scale), make_float2(__uint_as_float(now[2 * j]), __uint_as_float(now[2 * j + 1])), y);
                    }
                    if constexpr (kBias) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 u = sums[4 * i + j];
                            o[8 * i + 2 * j] = __ffma2_rn(make_float2(bias, bias), make_float2(u.x, u.y), o[8 * i + 2 * j]);
                            o[8 * i + 2 * j + 1] = __ffma2_rn(make_float2(bias, bias), make_float2(u.z, u.w), o[8 * i + 2 * j + 1]);
                        }
                    }
                }
                d.next();
                if (kBias && (q == kPer - 1 || g + 1 == g1)) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::kBarXEmpty + x.slot));
                    x.next();
                }
            }
            if (!alive) break;
            if (a.parts > 1) {
                // [column][row], where the activations and their sums were, once all warps have taken the last ones
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::kBarSums));
                alive = mbar_wait(bar(S::kBarSums), 0u);
                if (!alive) break;
                float* part_sums = reinterpret_cast<float*>(smem + S::kOffX) + 32 * quarter + lane;
#pragma unroll
                for (int j = 0; j < kCols; ++j) part_sums[(kCols * half + j) * kTcRows] = j & 1 ? o[j / 2].y : o[j / 2].x;
            } else if (n < a.N) {
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    if (m0 + j < a.M) {
                        float y = j & 1 ? o[j / 2].y : o[j / 2].x;
                        if (a.x_scales != nullptr) y *= __ldg(a.x_scales + m0 + j);
                        a.out[static_cast<size_t>(m0 + j) * a.N + n] = bf16_bits_rn(y);
                    }
                }
            }
        }
    }
    if (a.parts > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (warp >= 4 + kDecodeWarps) {
            const int m0 = tile0 % a.m_tiles * NB, n0 = tile0 / a.m_tiles * kTcRows;
            const int t = threadIdx.x - 32 * (4 + kDecodeWarps);
            const int row = t % kTcRows;
            float* mine = reinterpret_cast<float*>(smem + S::kOffX);
            for (int col = part * 2 + t / kTcRows; col < NB && m0 + col < a.M; col += 2 * a.parts) {
                float y = 0.0f;
                for (int r = 0; r < a.parts; ++r) y += cluster.map_shared_rank(mine, r)[col * kTcRows + row];
                if (a.x_scales != nullptr) y *= __ldg(a.x_scales + m0 + col);
                if (n0 + row < a.N) a.out[static_cast<size_t>(m0 + col) * a.N + n0 + row] = bf16_bits_rn(y);
            }
        }
        cluster.sync();                 // the others may still be reading this CTA's part
    }
    griddep_launch_dependents();
    fence_before();
    __syncthreads();
    if (warp == 3) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(512) : "memory");
    }
}

// Before the product: the sums of x over each group, [groups, m_pad], and 8-bit activations as bf16.
template <int G>
__global__ void __launch_bounds__(256) q4_prepare_kernel(const void* x, int eight, int M, int K, int m_pad, float* sums, uint16_t* x16) {
    constexpr int kLanes = G / 8;                 // of a group
    griddep_wait();
    const int blocks = K / 8;                     // of eight values, in a row
    const long long all = static_cast<long long>(M) * blocks, step = static_cast<long long>(gridDim.x) * 256;
    for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e - (threadIdx.x & 31) < all; e += step) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (e < all) v = q4_load_x(x, eight != 0, static_cast<size_t>(e) * 8);
        if (x16 != nullptr && e < all) *reinterpret_cast<uint4*>(x16 + static_cast<size_t>(e) * 8) = v;
        if (sums != nullptr) {
            float s = ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) +
                      ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            const int m = static_cast<int>(e / blocks), b = static_cast<int>(e - static_cast<long long>(m) * blocks);
            if (e < all && b % kLanes == 0) sums[static_cast<size_t>(b / kLanes) * m_pad + m] = s;
        }
    }
    griddep_launch_dependents();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Rows of `width` elements as boxes of 128 bytes x `rows`, swizzled; what lies outside is zero.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, int bytes, const void* p, int width, int height, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(height)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * bytes};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / bytes), static_cast<cuuint32_t>(rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, int NB, bool kBias>
cudaError_t launch_as(const TcArgs& args, const Q4Args& q, const void* x, const DeviceInfo& dev, cudaStream_t stream) {
    using S = TcShape<G, NB>;
    static std::atomic<unsigned long long> done{0};
    if (!smem_opt_in(q4_tc_kernel<G, NB, kBias>, S::kSmem, done)) return cudaErrorInvalidValue;
    CUtensorMap codes, xs;
    if (!make_map(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, q.codes, q.K / 8, q.N, kTcRows) ||
        !make_map(&xs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, q.K, q.M, NB))
        return cudaErrorInvalidValue;
    TcArgs a = args;
    a.m_tiles = (q.M + NB - 1) / NB;
    a.tiles = (q.N + kTcRows - 1) / kTcRows * a.m_tiles;
    // parts of k for clusters of CTAs, while all CTAs still run at once and each has two blocks of k or more
    const int blocks = (q.K + 2 * kTcStageK - 1) / (2 * kTcStageK);
    a.parts = 1;
    while (a.parts < 4 && 2 * a.parts * static_cast<long long>(a.tiles) <= dev.num_sms && blocks >= 4 * a.parts) a.parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.parts > 1 ? a.tiles * a.parts : (a.tiles < dev.num_sms ? a.tiles : dev.num_sms));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.parts; attr[1].val.clusterDim.y = 1; attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q4_tc_kernel<G, NB, kBias>, a, codes, xs);
}

template <int G, int NB>
cudaError_t launch_rows(const TcArgs& a, const Q4Args& q, const void* x, const DeviceInfo& dev, cudaStream_t stream) {
    return q.biases != nullptr ? launch_as<G, NB, true>(a, q, x, dev, stream) : launch_as<G, NB, false>(a, q, x, dev, stream);
}

// Activation rows of a tile: the one that leaves the fewest of them empty, the larger of two alike.
int tile_rows(int M) {
    if (M <= 32) return 32;
    if (M <= 64) return 64;
    const long long by128 = (M + 127ll) / 128 * 128, by192 = (M + 191ll) / 192 * 192;
    return by128 < by192 ? 128 : 192;
}

struct Workspace {
    size_t sums = 0, x16 = 0, total = 0;
    int m_pad = 0;
};
Workspace workspace_of(int M, int K, int groups, bool eight, bool bias) {
    constexpr size_t kCounters = size_t(1) << 20;      // the products' counters in front of a workspace stay zero
    Workspace w;
    w.m_pad = (M + tile_rows(M) - 1) / tile_rows(M) * tile_rows(M);
    size_t at = kCounters;
    w.sums = at;
    if (bias) at += (static_cast<size_t>(groups) * w.m_pad * 4 + 255) / 256 * 256;
    w.x16 = at;
    if (eight) at += static_cast<size_t>(M) * K * 2;
    w.total = bias || eight ? at : 0;
    return w;
}

template <int G>
cudaError_t launch_group(const Q4Args& q, char* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    const bool eight = q.x_scales != nullptr, bias = q.biases != nullptr;
    const Workspace w = workspace_of(q.M, q.K, q.groups, eight, bias);
    float* sums = bias ? reinterpret_cast<float*>(workspace + w.sums) : nullptr;
    uint16_t* x16 = eight ? reinterpret_cast<uint16_t*>(workspace + w.x16) : nullptr;
    if (eight || bias) {
        const long long ctas = (static_cast<long long>(q.M) * (q.K / 8) + 255) / 256, most = 8ll * dev.num_sms;
        const cudaError_t e = launch_programmatic(q4_prepare_kernel<G>, static_cast<unsigned>(ctas < most ? ctas : most), 256u, 0, stream,
                                                  q.x, eight ? 1 : 0, q.M, q.K, w.m_pad, sums, x16);
        if (e != cudaSuccess) return e;
    }
    TcArgs a = {};
    a.scales = q.scales; a.biases = q.biases; a.x_scales = q.x_scales; a.sums = sums; a.out = q.out;
    a.M = q.M; a.K = q.K; a.N = q.N; a.groups = q.groups; a.m_pad = w.m_pad;
    const void* x = eight ? static_cast<const void*>(x16) : q.x;
    switch (tile_rows(q.M)) {
        case 32: return launch_rows<G, 32>(a, q, x, dev, stream);
        case 64: return launch_rows<G, 64>(a, q, x, dev, stream);
        case 128: return launch_rows<G, 128>(a, q, x, dev, stream);
        default: return launch_rows<G, 192>(a, q, x, dev, stream);
    }
}

}  // namespace

size_t q4_tc_workspace_bytes(int M, int K, int groups, bool eight, bool bias) { return workspace_of(M, K, groups, eight, bias).total; }

cudaError_t launch_q4_tc(const Q4Args& q, int group, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    char* ws = static_cast<char*>(workspace);
    return group == 32 ? launch_group<32>(q, ws, dev, stream)
                       : group == 64 ? launch_group<64>(q, ws, dev, stream) : launch_group<128>(q, ws, dev, stream);
}

int q4_take_device_error(unsigned int* flags) {
    unsigned int v = 0u;
    if (cudaMemcpyFromSymbol(&v, g_q4_error, sizeof(v)) != cudaSuccess) return -5;
    if (v != 0u) {
        const unsigned int zero = 0u;
        if (cudaMemcpyToSymbol(g_q4_error, &zero, sizeof(zero)) != cudaSuccess) return -5;
    }
    *flags = v;
    return 0;
}

}  // namespace trellis
