// Products with 4-bit weights in groups, on the 5th-generation tensor cores.
//
//   D[n, m] (tensor memory, fp32) = sum_k w[n, k] x[m, k],   w = bf16(scale c + bias), or bf16(scale (c - 8))
//
// Each weight is rounded once to bf16, the type of its scale and of the activations (as the weights of the packed
// codes are): a code is a whole number of 4 bits, exact in bf16, and one multiply-add of bf16 pairs rounds the
// weight.  (Kept exact instead, with each group's sum scaled in fp32 on its way out of tensor memory, the
// product took 328 us at 2000 rows of K = 5120, N = 17408 in groups of 128, 1426 us in groups of 32 with
// biases; the group sums, not the products, were what it waited for.)
// That rounding is one of 2^-8 of the weight.  Where |bias| > 32 |scale| it would be more than 1% of what the codes
// say, and all of that in the end, so there a stage has two products: of
//   bf16(scale c + r), r = bias - o, o = bf16(bias + 8 scale), and of o, the same for all of a group,
// the second one's weights written when the first one is done.  To look at every group's scale and bias takes 0.3 us of 16.5 at one
// row, 0.8 of 20 at 64 rows in groups of 32, 235 us instead of 219 at 1999; with all groups far from zero those take 37, 42
// and 655 us, with one in 10000 28, 30 and 304.  |r| <= 16 |scale|, since bias is a bf16 number too, and r is one:
// both numbers are multiples of the last bit of the smaller, which is above 2^-8 of that, and so 2^-4 of the scale.
//
// A CTA's warps: one loads code tiles, one activation tiles, one issues the products, one keeps tensor
// memory, 4 load scales and biases, 16 turn codes into weights in tensor memory (the products' first operand), 4 store results
// (and widen 8-bit activations, where they are few).
// Tiles are 128 weight rows x NB activation rows; a CTA takes tile after tile (those of one block of weight rows
// next to each other, so that their codes come from L2), its results leaving while the next tile is under way.
// Where there are few tiles, a cluster of CTAs shares the k of one and adds its parts in shared memory, in order.
//
// Measured: 1999 rows, K = 5120, N = 17408 in groups of 128 205 us, 1.74 PFLOP/s, the tensor cores 86 to 89% busy; 64 rows in groups
// of 32 with biases 20.0 us, one row in groups of 64 with biases 16.5 us (3.0 TB/s): start, first tile and end take 4.5 us of it, the decode
// 2 beyond what the copies hide, the rest is the codes' way from cold memory to 136 SMs.  Weights made in registers for mma.sync
// instead, the k of a tile split over the warps of many small CTAs: 20 to 22 us at one row, 35 at 11 (here 21.3).
#include <cuda.h>
#include <cooperative_groups.h>
#include <mutex>

#include "kernels.h"
#include "kv_cache.cuh"
#include "trellis.h"
#include "trellis_device.cuh"

namespace trellis {

__device__ unsigned int g_q4_error = 0u;

namespace {

namespace cg = cooperative_groups;

constexpr int kRows = 128;                 // weight rows of a tile
constexpr int kStageK = 128;               // k of a stage
constexpr int kCodeBytes = kRows * 128;    // a code tile: 256 k (two stages) of 128 rows

constexpr int kDecodeWarps = 16, kStageWarps = 4;    // a stage's weights are made by four warps
constexpr int kStageGroups = kDecodeWarps / kStageWarps;
constexpr int kScaleWarps = 4, kScaleGroups = 16;    // 32 bytes of a row's scales (and of its biases) are loaded at once
constexpr int kStoreWarps = 4;
constexpr int kMostParts = 8;                       // of a tile's k, a CTA each
constexpr int kThreads = 32 * (4 + kDecodeWarps + kScaleWarps + kStoreWarps);

// Of tensor memory's 512 columns two D buffers take 2 NB, A slots of 64 the others.
template <int G, int NB>
struct Q4Shape {
    static constexpr int kA = NB == 128 ? 4 : 6;                    // stages under way: a slot of weights and one of activations each
    static constexpr int kXBytes = NB * kStageK * 2;              // two boxes of 64 k
    static constexpr int kPer = kStageK / G;                        // groups of a stage
    static constexpr int kScaleStages = kScaleGroups / kPer;        // stages of a run of scales
    static constexpr int kScaleBytes = kRows * kScaleGroups * 4, kScale = 2;
    static constexpr int kOffX = 0, kOffScale = kA * kXBytes, kOffCode = kOffScale + kScale * kScaleBytes;
    static constexpr int kCode = 4;                                 // code tiles under way (6 and 8 take 0.3 to 0.7 us more: the first ones come later)
    static constexpr int kOffOffset = kOffCode + kCode * kCodeBytes;    // bf16, of groups far from zero
    static constexpr int kOffBar = kOffOffset + kScale * kRows * kScaleGroups * 2;
    static constexpr int kBarFull = 0, kBarEmpty = kA, kBarCode = 2 * kA, kBarCodeEmpty = kBarCode + kCode;
    static constexpr int kBarD = kBarCodeEmpty + kCode, kBarDEmpty = kBarD + 2;
    static constexpr int kBarScale = kBarDEmpty + 2, kBarScaleEmpty = kBarScale + kScale;
    // a stage's second product: the first one is done, the second one's weights are there (one of each for the warps that made them)
    static constexpr int kBarFirst = kBarScaleEmpty + kScale, kBarSecond = kBarFirst + kStageGroups, kBars = kBarSecond + kStageGroups;
    // Of a run of scales: whether groups lie far from zero, a byte for 32 rows.  The products read it after the run's slot went to
    // others, kA stages after the weights were made at most, which is up to three runs of two stages: with the two slots' five.
    static constexpr int kFarRing = 8, kOffFar = kOffBar + 8 * kBars;
    static constexpr int kOffTaddr = kOffFar + kFarRing * 4;
    static constexpr int kSmem = kOffTaddr + 16 + 1024;             // the base is rounded up to 1 KB
    static constexpr uint32_t kInstr = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NB >> 3) << 17) |
                                       (static_cast<uint32_t>(kRows >> 4) << 24);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    static constexpr int kAColumn = 512 - 64 * kA;
    static_assert(2 * NB <= kAColumn, "tensor memory");
    static_assert(kRows * NB * 4 <= kOffBar, "a part of the sums fits where operands were");
};

struct Q4Args {
    const uint32_t* codes;          // [N, K / 8]
    const uint16_t *scales, *biases;  // bf16 [N, groups]; biases may be NULL
    const float* x_scales;          // [M], or NULL
    const uint8_t* x8;              // e4m3 [M, K], where they are widened on their way to shared memory
    uint16_t* out;                  // bf16 [M, N]
    int M, K, N, groups;
    int m_tiles, tiles, parts;
};

// ---- waits --------------------------------------------------------------------------
// Every wait is bounded, as the other tensor-core kernels' are: one that runs out sets the error word and its
// warp leaves its loops; copies in flight are waited for, tensor memory is given back.
constexpr unsigned long long kWaitNs = 2000000000ull;   // 2 s
constexpr uint32_t kWaitPollCap = 1u << 26, kPollNs = 1000000u;

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_many(uint32_t bar, int count) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(count) : "memory");
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
// A poll may sleep for as long as its hint: without one a waiting warp comes back often, and the polls of those that wait
// for most of a tile took issue slots from those that make its weights.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t i = 0; i < kWaitPollCap; ++i) {
        uint32_t ok;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.b32 %0, 1, 0, p;\n}"
                     : "=r"(ok) : "r"(bar), "r"(parity), "r"(kPollNs) : "memory");
        if (ok != 0u) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > kWaitNs) break;
    }
    atomicOr(&g_q4_error, 1u);
    return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    return mbar_try(bar, parity) || mbar_wait_long(bar, parity);
}
// For a whole warp whose lanes go on together, or none does: a wait may run out for some of them only, and those that were left
// would meet another warp barrier, or arrive for the others.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
// K-major, 128-byte swizzle: 1 KB between atoms of 8 rows, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}
// One product of 16 k, its operands a base and an immediate (a shared-memory offset only reaches the address field).
template <int kOffA, int kOffB>
__device__ __forceinline__ void mma_step(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, uint32_t accumulate, uint32_t elected) {
    asm volatile("{\n .reg .pred p, e;\n .reg .b64 y;\n .reg .b32 x;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %7, 0;\n"
                 " add.s32 x, %1, %5;\n add.s64 y, %2, %6;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(instr), "r"(accumulate), "n"(kOffA), "n"(kOffB >> 4), "r"(elected) : "memory");
}
// A stage's eight products, added to the sum or (the first one of a tile) begun anew.
template <int NB, int k = 0>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, uint32_t accumulate, uint32_t elected) {
    mma_step<8 * k, (k >> 2) * (NB * 128) + (k & 3) * 32>(d, a, b, instr, k > 0 ? 1u : accumulate, elected);
    if constexpr (k + 1 < kStageK / 16) mma_stage<NB, k + 1>(d, a, b, instr, accumulate, elected);
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t elected) {
    asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
                 :: "r"(bar), "r"(elected) : "memory");
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// From 1/4 up: the weights of a word's codes 2i and 2i + 1 as bf16 pairs, i = 0 .. 3.  Even and odd codes are masked into the bytes of
// two words, and one byte permutation a pair puts a code into the low byte of each half (the upper bytes are copies of the
// sign of a byte that has none).  Such a half is the bf16 number c 2^-133, below the normal ones: multiplied by 2^127 it
// is c 2^-6, exactly, less 8 2^-6 without biases; and 64 times the scale makes the weight in one rounding.
template <bool kBias>
__device__ __forceinline__ void weights_of(uint32_t w, uint32_t scale64, uint32_t bias, uint32_t* p) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(c) : "r"(even), "r"(odd), "r"(0xc480u + 0x1111u * static_cast<uint32_t>(i)));
        if constexpr (kBias) {
            uint32_t v;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(c), "r"(0x7f007f00u));
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(p[i]) : "r"(v), "r"(scale64), "r"(bias));
        } else {
            uint32_t v;
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(c), "r"(0x7f007f00u), "r"(0xbe00be00u));
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(v), "r"(scale64));
        }
    }
}
// The same where scales are below 1/4, as those of a layer's weights are: a code three bits further up is c 2^-130, its product with
// 2^130 of the scale is added to the bias (without biases to -8 times the scale, which is exact) in one rounding of the same number.
// 12 instructions for eight weights, where the other takes 15: 0.4 us of 16.5 at one row, 0.6 of 20 at 64, 2.5 of 235 at 1999
// in groups of 32.
__device__ __forceinline__ void weights_below(uint32_t w, uint32_t scale130, uint32_t bias, uint32_t* p) {
    const uint32_t even = (w << 3) & 0x78787878u, odd = (w >> 1) & 0x78787878u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c;
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(c) : "r"(even), "r"(odd), "r"(0xc480u + 0x1111u * static_cast<uint32_t>(i)));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(p[i]) : "r"(c), "r"(scale130), "r"(bias));
    }
}
// Pairs times a power of two.
__device__ __forceinline__ uint32_t times(uint32_t v, uint32_t factor) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(factor));
    return r;
}
// 64 times the bf16 number in the low half, in both halves.
__device__ __forceinline__ uint32_t scale64_of(uint32_t v) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(v, 0u, 0x1010)), "r"(0x42804280u));
    return r;
}

// A group's scale and, above it, its bias: whether the bias is far from zero, and its part that is left to the second product.
// Groups of one value (scale 0) are exact as they are; next to the largest number, and where a bias is no number, nothing is parted.
__device__ __forceinline__ bool is_far(uint32_t sb) {
    const float s = fabsf(__uint_as_float(sb << 16)), b = fabsf(__uint_as_float(sb & 0xffff0000u));
    return b > 32.0f * s && s > 0.0f && b < 8.507059173023462e37f;         // 2^126
}
// A bound that takes three instructions: |bias|'s bits less |scale|'s, above those of the scale.  Bits count as the logarithm does, 128 for
// a factor of two, but for 0.086 of that at most, so a far one is never below 5 * 128 - 12.
constexpr int kNearly = (5 * 128 - 12) << 16;
__device__ __forceinline__ int distance_of(uint32_t sb) { return static_cast<int>((sb & 0x7fff7fffu) * (1u - 65536u)); }
__device__ __forceinline__ uint32_t offset_of(uint32_t sb) {               // in both halves
    uint32_t o;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o) : "r"(__byte_perm(sb, 0u, 0x1010)), "r"(0x41004100u), "r"(__byte_perm(sb, 0u, 0x3232)));
    return is_far(sb) ? o : 0u;
}
// The group as the first product has it: its bias less that.
__device__ __forceinline__ uint32_t without_offset(uint32_t sb, uint32_t offset) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(sb, 0u, 0x3232)), "r"(offset));
    return __byte_perm(sb, r, 0x5410);
}

// Eight e4m3 codes as bf16, exactly.
__device__ __forceinline__ uint4 widened(uint2 v) {
    uint32_t f[4], r[4];
    e4m3x4_to_f16x2(v.x, f[0], f[1]);
    e4m3x4_to_f16x2(v.y, f[2], f[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 d = f16x2_to_f32(f[i]);
        r[i] = pack_bf16x2(d.x, d.y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Where group g of a row's sixteen stands: fours of them are turned by the row.
__device__ __forceinline__ int scale_column(int row, int g) { return g ^ (((row >> 1) & 3) << 2); }

template <int G, int NB, bool kBias, bool kEight>
__global__ void __launch_bounds__(kThreads, 1)
q4_kernel(const __grid_constant__ Q4Args a, const __grid_constant__ CUtensorMap code_map, const __grid_constant__ CUtensorMap x_map) {
    using S = Q4Shape<G, NB>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    unsigned char* const smem = smem_raw + (sbase - sraw);
    auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kA; ++i) {
            // weights by the warps that made them, activations by their bytes or by the warps that widened them
            mbar_init(bar(S::kBarFull + i), kStageWarps + (kEight ? kStoreWarps : 1));
            mbar_init(bar(S::kBarEmpty + i), 1);
        }
        for (int i = 0; i < S::kCode; ++i) {
            mbar_init(bar(S::kBarCode + i), 1);
            mbar_init(bar(S::kBarCodeEmpty + i), 2 * kStageWarps);       // two stages
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(S::kBarD + i), 1);
            mbar_init(bar(S::kBarDEmpty + i), kStoreWarps);
        }
        for (int i = 0; i < S::kScale; ++i) {
            mbar_init(bar(S::kBarScale + i), kScaleWarps);
            mbar_init(bar(S::kBarScaleEmpty + i), kStageWarps * S::kScaleStages);
        }
        for (int i = 0; i < kStageGroups; ++i) {
            mbar_init(bar(S::kBarFirst + i), 1);
            mbar_init(bar(S::kBarSecond + i), kStageWarps);
        }
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
    const uint32_t t_a = taddr + S::kAColumn;

    // this CTA's share of k, in blocks of two stages, and its first tile
    const int part = a.parts > 1 ? static_cast<int>(blockIdx.x) % a.parts : 0;
    const int blocks = (a.K + 2 * kStageK - 1) / (2 * kStageK);
    const int b0 = static_cast<int>(static_cast<long long>(blocks) * part / a.parts);
    const int b1 = static_cast<int>(static_cast<long long>(blocks) * (part + 1) / a.parts);
    const int s0 = 2 * b0, s1 = 2 * b1;         // past K: codes, scales and activations of zero
    const int tile0 = a.parts > 1 ? static_cast<int>(blockIdx.x) / a.parts : static_cast<int>(blockIdx.x);
    const int tile_step = a.parts > 1 ? a.tiles : static_cast<int>(gridDim.x);
    if (warp == 0 && lane == 0) {
        // L2 prefetches only: nothing reaches the CTA before the wait for the previous grid
        for (int b = b0; b < b1 && b < b0 + S::kCode; ++b)
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                         :: "l"(reinterpret_cast<uint64_t>(&code_map)), "r"(b * 32), "r"(tile0 / a.m_tiles * kRows) : "memory");
    }
    if (warp >= 4 + kDecodeWarps && warp < 4 + kDecodeWarps + kScaleWarps) {
        // a row's first 256 bytes of scales and of biases (one row 16.9 -> 16.6 us, 64 rows in groups of 32 21.6 -> 20.7; all of them, or the
        // first 32 bytes alone, 0.3 to 0.5 more)
        const int n = min(tile0 / a.m_tiles * kRows + 32 * (warp - 4 - kDecodeWarps) + lane, a.N - 1);
        const size_t at = static_cast<size_t>(n) * a.groups;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = s0 * S::kPer + 64 * i;
            if (g < a.groups) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.scales + at + g));
            if (kBias && g < a.groups) asm volatile("prefetch.global.L2 [%0];" :: "l"(a.biases + at + g));
        }
    }
    griddep_wait();
    // The next grid may set itself up where an SM has no tile of this one (whose CTAs take all of tensor memory, and nearly all
    // registers); it waits for this one's end before it reads.
    griddep_launch_dependents();

    // Slots are taken in turn: use number i of a ring of n is slot i % n, its phase's parity (i / n) & 1.  A parity tells a
    // phase only from its neighbours, so whoever waits for use i has to know that use i - n is over.  The decoding warps,
    // which meet every fourth stage only, do because a tile has an even number of them: they meet every second code tile
    // (of a ring of four), and go on by two runs of scales at most (of a ring of two, which is filled in order).  Of the ring of
    // operand slots a group has waited for the stage four before, four or six slots back from there; that the use before the one
    // it waits for is over, it knows because commits arrive in the order of their products.
    bool alive = true;
    if (warp == 0) {
        // ---------------------------------------------------------------- code tiles
        if (lane == 0) {
            uint32_t i = 0;
            for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
                const int n0 = tile / a.m_tiles * kRows;
                for (int b = b0; b < b1; ++b, ++i) {
                    const uint32_t slot = i % S::kCode;
                    alive = mbar_wait(bar(S::kBarCodeEmpty + slot), ((i / S::kCode) & 1u) ^ 1u);
                    if (!alive) break;
                    mbar_expect(bar(S::kBarCode + slot), kCodeBytes);
                    tma_load_2d(sbase + S::kOffCode + slot * kCodeBytes, &code_map, b * 32, n0, bar(S::kBarCode + slot));
                }
            }
            // what was asked for has landed before the CTA ends
            for (uint32_t j = i > S::kCode ? i - S::kCode : 0u; j < i; ++j) (void)mbar_wait(bar(S::kBarCode + j % S::kCode), (j / S::kCode) & 1u);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- activation tiles
        if (!kEight && lane == 0) {
            uint32_t i = 0;
            for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
                const int m0 = tile % a.m_tiles * NB;
                for (int s = s0; s < s1; ++s, ++i) {
                    const uint32_t slot = i % S::kA, full = bar(S::kBarFull + slot), dst = sbase + S::kOffX + slot * S::kXBytes;
                    alive = mbar_wait(bar(S::kBarEmpty + slot), ((i / S::kA) & 1u) ^ 1u);
                    if (!alive) break;
                    mbar_expect(full, S::kXBytes);
                    tma_load_2d(dst, &x_map, s * kStageK, m0, full);
                    tma_load_2d(dst + NB * 128, &x_map, s * kStageK + 64, m0, full);
                }
            }
            // (a stage whose weights were never made keeps its barrier: that wait gives up)
            for (uint32_t j = i > S::kA ? i - S::kA : 0u; j < i; ++j) (void)mbar_wait(bar(S::kBarFull + j % S::kA), (j / S::kA) & 1u);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- products
        // All lanes walk the same path and one issues, so that the operands live in uniform registers.
        const uint32_t elected = elect_lane();
        const uint64_t desc0 = smem_desc(sbase + S::kOffX);
        uint32_t slot = 0, turn = 0, d = 0;
        uint32_t group = 0, seconds = 0;            // of the warps that made the stage, and their second products' parities
        uint32_t runs_before = 0;
        const uint32_t runs = (s1 - s0 + S::kScaleStages - 1) / S::kScaleStages;
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step, ++d, runs_before += runs) {
            const uint32_t td = taddr + (d & 1u) * NB;
            alive = mbar_wait_warp(bar(S::kBarDEmpty + (d & 1u)), ((d >> 1) & 1u) ^ 1u);
            for (int s = s0; s < s1 && alive; ++s) {
                alive = mbar_wait_warp(bar(S::kBarFull + slot), turn);
                if (!alive) break;
                fence_after();
                mma_stage<NB>(td, t_a + slot * 64, desc0 + static_cast<uint64_t>(slot * (S::kXBytes >> 4)), S::kInstr, s > s0 ? 1u : 0u, elected);
                if constexpr (kBias) {
                    const uint32_t run = runs_before + static_cast<uint32_t>(s - s0) / S::kScaleStages;
                    if (__any_sync(0xffffffffu, lds32(sbase + S::kOffFar + run % S::kFarRing * 4) != 0u)) {
                        mma_commit(bar(S::kBarFirst + group), elected);
                        alive = mbar_wait_warp(bar(S::kBarSecond + group), (seconds >> group) & 1u);
                        if (!alive) break;
                        seconds ^= 1u << group;
                        fence_after();
                        mma_stage<NB>(td, t_a + slot * 64, desc0 + static_cast<uint64_t>(slot * (S::kXBytes >> 4)), S::kInstr, 1u, elected);
                    }
                    group = (group + 1) % kStageGroups;
                }
                mma_commit(bar(S::kBarEmpty + slot), elected);
                if (++slot == S::kA) { slot = 0; turn ^= 1u; }
            }
            // also where a wait gave up: what was issued is done before tensor memory is given back
            mma_commit(bar(S::kBarD + (d & 1u)), elected);
        }
        if (d > 0) (void)mbar_wait(bar(S::kBarD + ((d - 1) & 1u)), ((d - 1) >> 1) & 1u);
    } else if (warp >= 4 && warp < 4 + kDecodeWarps) {
        // ---------------------------------------------------------------- codes to weights
        // 32 rows (a lane's row is its lane of tensor memory) of every fourth stage
        constexpr int kGroups = kStageGroups;
        static_assert(S::kA >= kGroups, "a slot for each four warps");
        const int quarter = warp & 3, group = (warp - 4) >> 2;
        const int row = 32 * quarter + lane;
        const uint32_t t_row = t_a + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t row_at = sbase + S::kOffCode + row * 128, turned = static_cast<uint32_t>(row & 7) << 4;
        constexpr int kPer = S::kPer;
        uint32_t slot = group, parity = 1u;                          // of its next stage
        uint32_t firsts = 0;                                         // parity of its next stage with two products
        int ahead = group;                                           // stages from this tile's first to it
        uint32_t blocks_before = 0, runs_before = 0;
        const uint32_t runs = (s1 - s0 + S::kScaleStages - 1) / S::kScaleStages;
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step, ahead -= s1 - s0, blocks_before += b1 - b0, runs_before += runs) {
            int s = s0 + ahead;
            for (; s < s1; s += kGroups) {
                const uint32_t b_i = blocks_before + static_cast<uint32_t>((s - s0) >> 1), code = b_i % S::kCode;
                const uint32_t run = runs_before + static_cast<uint32_t>(s - s0) / S::kScaleStages, run_slot = run % S::kScale;
                alive = mbar_wait(bar(S::kBarCode + code), (b_i / S::kCode) & 1u) && mbar_wait(bar(S::kBarScale + run_slot), (run / S::kScale) & 1u);
                // scale, and bias above it, of each of the stage's groups; a row's are turned so that the rows of a quarter
                // warp lie in different banks
                uint32_t v[kPer];
                const uint32_t scale_at = sbase + S::kOffScale + run_slot * S::kScaleBytes + row * (kScaleGroups * 4) +
                                          scale_column(row, static_cast<int>(static_cast<uint32_t>(s - s0) % S::kScaleStages * kPer)) * 4;
                if constexpr (kPer == 4) {
                    const uint4 u = lds128(scale_at);
                    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
                } else if constexpr (kPer == 2) {
                    asm volatile("ld.volatile.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(scale_at));
                } else {
                    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(scale_at));
                }
                const uint32_t at = row_at + code * kCodeBytes + ((s & 1) << 6);
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = lds128(at ^ (turned ^ (16 * j)));
                const uint32_t far = kBias ? lds32(sbase + S::kOffFar + run % S::kFarRing * 4) : 0u;
                // what follows needs all lanes: they go on, or none does
                alive = __all_sync(0xffffffffu, alive && mbar_wait(bar(S::kBarEmpty + slot), parity));
                if (!alive) break;
                fence_after();
                const uint32_t to = t_row + slot * 64;
                uint32_t most = 0u;
#pragma unroll
                for (int j = 0; j < kPer; ++j) most = max(most, v[j] & 0x7fffu);
                const bool below = __all_sync(0xffffffffu, most < 0x3e80u);      // magnitudes below 1/4
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t sb = v[j * kPer / 4];
                    uint32_t p[16];
                    if (below) {
                        const uint32_t s = __byte_perm(sb, 0u, 0x1010), scale = times(times(s, 0x60006000u), 0x60006000u);
                        const uint32_t bias = kBias ? __byte_perm(sb, 0u, 0x3232) : times(s, 0xc100c100u);
                        weights_below(w[j].x, scale, bias, p); weights_below(w[j].y, scale, bias, p + 4);
                        weights_below(w[j].z, scale, bias, p + 8); weights_below(w[j].w, scale, bias, p + 12);
                    } else {
                        const uint32_t scale = scale64_of(sb), bias = kBias ? __byte_perm(sb, 0u, 0x3232) : 0u;
                        weights_of<kBias>(w[j].x, scale, bias, p); weights_of<kBias>(w[j].y, scale, bias, p + 4);
                        weights_of<kBias>(w[j].z, scale, bias, p + 8); weights_of<kBias>(w[j].w, scale, bias, p + 12);
                    }
                    tmem_st16(to + 16 * j, p);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (far != 0u) {                     // of any of the 128 rows
                    if (lane == 0) mbar_arrive(bar(S::kBarFull + slot));
                    alive = mbar_wait_warp(bar(S::kBarFirst + group), firsts);
                    if (!alive) break;
                    firsts ^= 1u;
                    fence_after();
                    // offsets stand only where some of these 32 rows have one
                    const uint32_t mine = (far >> (8 * quarter)) & 1u ? 0x10001u : 0u;
                    const volatile uint16_t* offsets = reinterpret_cast<const volatile uint16_t*>(smem + S::kOffOffset) + (run_slot * kRows + row) * kScaleGroups;
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t o = offsets[scale_column(row, static_cast<int>(static_cast<uint32_t>(s - s0) % S::kScaleStages * kPer) + j * kPer / 4)] * mine;
                        const uint32_t p[16] = {o, o, o, o, o, o, o, o, o, o, o, o, o, o, o, o};
                        tmem_st16(to + 16 * j, p);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    fence_before();
                    __syncwarp();
                }
                // Codes and scales make room only now that the weights made of them are stored, so that their loads are known to
                // be over: given back right after the loads were issued, now and then they were those of the next tile in the slot.
                if (lane == 0) {
                    mbar_arrive(far != 0u ? bar(S::kBarSecond + group) : bar(S::kBarFull + slot));
                    mbar_arrive(bar(S::kBarScaleEmpty + run_slot));
                    mbar_arrive(bar(S::kBarCodeEmpty + code));
                }
                slot += kGroups;
                if (slot >= S::kA) { slot -= S::kA; parity ^= 1u; }
            }
            ahead = s - s0;
        }
    } else if (warp >= 4 + kDecodeWarps && warp < 4 + kDecodeWarps + kScaleWarps) {
        // ---------------------------------------------------------------- scales and biases
        // Sixteen lanes a row, 32 bytes (a lane a row, stage by stage as the codes are taken, looks up 32 lines for 64 bytes and
        // fetches each sector again and again).  A run's loads are under way while those of the one before are used.
        constexpr int kLoads = 16;                                   // of two rows each
        const int first_row = 32 * (warp - 4 - kDecodeWarps) + (lane >> 4), of = lane & 15;
        const int runs = (s1 - s0 + S::kScaleStages - 1) / S::kScaleStages;
        uint32_t i = 0, v[kLoads];
        auto load = [&](int tile, int run) {
            const int g = s0 * S::kPer + run * kScaleGroups + of;
            const bool has = g < a.groups;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int n = min(tile / a.m_tiles * kRows + first_row + 2 * j, a.N - 1);
                const size_t at = static_cast<size_t>(n) * a.groups + g;
                v[j] = has ? __ldg(a.scales + at) : 0u;
                if constexpr (kBias) v[j] |= has ? static_cast<uint32_t>(__ldg(a.biases + at)) << 16 : 0u;
            }
        };
        if (tile0 < a.tiles) load(tile0, 0);
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step) {
            for (int run = 0; run < runs; ++run, ++i) {
                const uint32_t slot = i % S::kScale;
                bool far = false;
                if constexpr (kBias) {
                    int most[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) most[j % 4] = max(most[j % 4], distance_of(v[j]));
                    far = __any_sync(0xffffffffu, max(max(most[0], most[1]), max(most[2], most[3])) >= kNearly);
                }
                alive = mbar_wait_warp(bar(S::kBarScaleEmpty + slot), ((i / S::kScale) & 1u) ^ 1u);
                if (!alive) break;
                if constexpr (kBias) {
                    if (far) {
                        uint16_t* offsets = reinterpret_cast<uint16_t*>(smem + S::kOffOffset) + slot * kRows * kScaleGroups;
#pragma unroll
                        for (int j = 0; j < kLoads; ++j) {
                            const int r = first_row + 2 * j;
                            const uint32_t o = offset_of(v[j]);
                            offsets[r * kScaleGroups + scale_column(r, of)] = static_cast<uint16_t>(o);
                            v[j] = without_offset(v[j], o);
                        }
                    }
                    if (lane == 0) smem[S::kOffFar + i % S::kFarRing * 4 + warp - 4 - kDecodeWarps] = far;
                }
                uint32_t* to = reinterpret_cast<uint32_t*>(smem + S::kOffScale + slot * S::kScaleBytes);
#pragma unroll
                for (int j = 0; j < kLoads; ++j) {
                    const int r = first_row + 2 * j;
                    to[r * kScaleGroups + scale_column(r, of)] = v[j];
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(S::kBarScale + slot));
                    // for the stages that a tile's last run does not have
                    const int missing = (run + 1) * S::kScaleStages - (s1 - s0);
                    if (missing > 0 && warp == 4 + kDecodeWarps) mbar_arrive_many(bar(S::kBarScaleEmpty + slot), kStageWarps * missing);
                }
                const bool more = run + 1 < runs;
                if (more || tile + tile_step < a.tiles) load(more ? tile : tile + tile_step, more ? run + 1 : 0);
            }
        }
    } else if (warp >= 4 + kDecodeWarps + kScaleWarps) {
        // ---------------------------------------------------------------- results, and before them 8-bit activations
        const int quarter = warp & 3;
        constexpr int kStep = NB < 32 ? 16 : 32;
        uint32_t d = 0;
        // Sixteen codes a thread and 16 activation rows, some stages ahead.
        constexpr int kPieces = kEight ? NB / 16 : 1, kFar = 3;
        const int x_row = (32 * (warp - 4 - kDecodeWarps - kScaleWarps) + lane) >> 3, x_chunk = lane & 7;
        uint4 x8[kFar][kPieces];
        uint32_t x_slot = 0, x_turn = 1u;
        auto load = [&](int s, uint4 (&v)[kPieces]) {
            const int k = s * kStageK + 16 * x_chunk;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int m = x_row + 16 * i;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (s < s1 && k < a.K && m < a.M) v[i] = *reinterpret_cast<const uint4*>(a.x8 + static_cast<size_t>(m) * a.K + k);
            }
        };
        for (int tile = tile0; tile < a.tiles && alive; tile += tile_step, ++d) {
            const int m0 = tile % a.m_tiles * NB, n = tile / a.m_tiles * kRows + 32 * quarter + lane;
            if constexpr (kEight) {
#pragma unroll
                for (int f = 0; f < kFar; ++f) load(s0 + f, x8[f]);
                for (int s = s0; s < s1; s += kFar) {
#pragma unroll
                    for (int f = 0; f < kFar; ++f) {
                        if (s + f >= s1) break;
                        // No lane leaves before the vote below, so that all meet at the warp barrier; one whose wait ran out waits no
                        // more (a vote here: 11 rows 21.2 -> 21.6 us).
                        alive &= mbar_try(bar(S::kBarEmpty + x_slot), x_turn) || (alive && mbar_wait_long(bar(S::kBarEmpty + x_slot), x_turn));
                        // where the tensor copies put bf16 tiles: boxes of 64 k, rows of 128 bytes, their pieces of 16 turned by the row
                        const uint32_t to = sbase + S::kOffX + x_slot * S::kXBytes + (x_chunk >> 2) * (NB * 128);
#pragma unroll
                        for (int i = 0; i < kPieces; ++i) {
                            const int m = x_row + 16 * i;
                            const uint4 lo = widened(make_uint2(x8[f][i].x, x8[f][i].y)), hi = widened(make_uint2(x8[f][i].z, x8[f][i].w));
                            sts128(to + m * 128 + (((2 * (x_chunk & 3)) ^ (m & 7)) << 4), lo);
                            sts128(to + m * 128 + (((2 * (x_chunk & 3) + 1) ^ (m & 7)) << 4), hi);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(S::kBarFull + x_slot));
                        if (++x_slot == S::kA) { x_slot = 0; x_turn ^= 1u; }
                        load(s + f + kFar, x8[f]);
                    }
                }
            }
            const uint32_t t_row = taddr + (static_cast<uint32_t>(32 * quarter) << 16) + (d & 1u) * NB;
            alive = __all_sync(0xffffffffu, alive && mbar_wait(bar(S::kBarD + (d & 1u)), (d >> 1) & 1u));       // as the decoding warps
            if (!alive) break;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < NB; c += kStep) {
                uint32_t v[kStep / 16][16];
#pragma unroll
                for (int i = 0; i < kStep / 16; ++i) tmem_ld16(v[i], t_row + c + 16 * i);
#pragma unroll
                for (int i = 0; i < kStep / 16; ++i) tmem_wait_ld(v[i]);
                if (c + kStep == NB) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::kBarDEmpty + (d & 1u)));
                }
                if (a.parts > 1) {
                    // [column][row], where the operands were: all of the products are done
                    float* part_sums = reinterpret_cast<float*>(smem) + c * kRows + 32 * quarter + lane;
#pragma unroll
                    for (int j = 0; j < kStep; ++j) part_sums[j * kRows] = __uint_as_float(v[j / 16][j % 16]);
                } else {
                    if (a.x_scales != nullptr) {
                        const float s = lane < kStep && m0 + c + lane < a.M ? a.x_scales[m0 + c + lane] : 0.0f;
#pragma unroll
                        for (int j = 0; j < kStep; ++j)
                            v[j / 16][j % 16] = __float_as_uint(__uint_as_float(v[j / 16][j % 16]) * __shfl_sync(0xffffffffu, s, j));
                    }
                    // all of the rows that there are, without a branch between two stores
                    const int rows = n < a.N ? a.M - m0 - c : 0;
                    uint16_t* to = a.out + static_cast<size_t>(m0 + c) * a.N + n;
#pragma unroll
                    for (int j = 0; j < kStep; ++j, to += a.N)
                        if (j < rows) *to = bf16_bits_rn(__uint_as_float(v[j / 16][j % 16]));
                }
            }
        }
    }
    __syncwarp();
    if (a.parts > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int m0 = tile0 % a.m_tiles * NB, n0 = tile0 / a.m_tiles * kRows;
        // a warp a column, four rows a lane; all parts are on their way before the first is added
        constexpr int kWarps = kThreads / 32;
        const int row = 4 * lane;
        const bool wide = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
        const float* mine = reinterpret_cast<const float*>(smem) + row;
        for (int col = part * kWarps + warp; col < NB && m0 + col < a.M; col += kWarps * a.parts) {
            float4 of[kMostParts];
#pragma unroll
            for (int r = 0; r < kMostParts; ++r)
                if (r < a.parts) of[r] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(mine, r) + col * kRows);
            const float s = a.x_scales != nullptr ? a.x_scales[m0 + col] : 1.0f;
            float4 y = of[0];
#pragma unroll
            for (int r = 1; r < kMostParts; ++r)
                if (r < a.parts) y.x += of[r].x, y.y += of[r].y, y.z += of[r].z, y.w += of[r].w;
            uint16_t* to = a.out + static_cast<size_t>(m0 + col) * a.N + n0 + row;
            if (wide) {
                if (n0 + row < a.N) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(y.x * s, y.y * s), pack_bf16x2(y.z * s, y.w * s));
            } else {
                const float v[4] = {y.x * s, y.y * s, y.z * s, y.w * s};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + row + i < a.N) to[i] = bf16_bits_rn(v[i]);
            }
        }
        cluster.sync();                 // the others may still be reading this CTA's part
    }
    fence_before();
    __syncthreads();
    if (warp == 3) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(512) : "memory");
    }
}

// Before a product of more rows: 8-bit activations as bf16.
__global__ void __launch_bounds__(256) q4_widen_kernel(const uint8_t* x, long long count, uint16_t* x16) {
    griddep_wait();
    for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < count; e += static_cast<long long>(gridDim.x) * 256)
        *reinterpret_cast<uint4*>(x16 + e * 8) = widened(reinterpret_cast<const uint2*>(x)[e]);
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

template <int G, int NB, bool kBias, bool kEight>
cudaError_t launch_as(Q4Args a, const void* x, const DeviceInfo& dev, cudaStream_t stream) {
    using S = Q4Shape<G, NB>;
    static std::atomic<unsigned long long> done{0};
    if (!smem_opt_in(q4_kernel<G, NB, kBias, kEight>, S::kSmem, done)) return cudaErrorInvalidValue;
    CUtensorMap codes, xs;
    if (!make_map(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.codes, a.K / 8, a.N, kRows)) return cudaErrorInvalidValue;
    if (kEight)
        xs = codes;             // not used
    else if (!make_map(&xs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, a.K, a.M, NB))
        return cudaErrorInvalidValue;
    a.m_tiles = (a.M + NB - 1) / NB;
    a.tiles = (a.N + kRows - 1) / kRows * a.m_tiles;
    // Parts of k for clusters of CTAs, while all CTAs still run at once.  The join takes about 2 us, of 128 rows more, so each part
    // has two blocks of k or more (one row, K = 2048, N = 1024 in four parts 5.8 us, in one 7.8), of 128 rows five (512 rows, K = 2048,
    // N = 1024 in two parts 10.6 us, in one 9.9; K = 5120 in four 13.0, in two 14.3), and K up to 1280 is not split (64 rows, K =
    // N = 1024 in two parts 7.8 us, in one 6.1).  Clusters of more than four are placed less densely: half of the SMs (one row, K =
    // 5120, N = 2560 in four parts 8.8 us, in seven 13.1).
    const int blocks = (a.K + 2 * kStageK - 1) / (2 * kStageK), least = NB == 128 ? 5 : 2;
    a.parts = 1;
    while (a.parts < kMostParts && (a.parts + 1ll) * a.tiles <= (a.parts < 4 ? dev.num_sms : dev.num_sms / 2) && blocks >= 6 &&
           blocks >= least * (a.parts + 1))
        ++a.parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.parts > 1 ? a.tiles * a.parts : (a.tiles < dev.num_sms ? a.tiles : dev.num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.parts; attr[1].val.clusterDim.y = 1; attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_kernel<G, NB, kBias, kEight>, a, codes, xs);
}

// 8-bit activations of up to 32 rows are widened in the product itself; of more, every tile of weight rows would widen them
// again, so a kernel before it does (1 row, K = 5120, N = 17408 18.8 -> 17.8 us, N = 5120 12.0 -> 10.5; 11 rows, K = 17408,
// N = 5120 21.9 -> 21.8; 32 rows in groups of 32 23.9 -> 23.4; and one launch less).
constexpr int kWidenRows = 32;

template <int G, int NB>
cudaError_t launch_rows(const Q4Args& a, const void* x, const DeviceInfo& dev, cudaStream_t stream) {
    if constexpr (NB <= kWidenRows)
        if (a.x8 != nullptr)
            return a.biases != nullptr ? launch_as<G, NB, true, true>(a, x, dev, stream) : launch_as<G, NB, false, true>(a, x, dev, stream);
    return a.biases != nullptr ? launch_as<G, NB, true, false>(a, x, dev, stream) : launch_as<G, NB, false, false>(a, x, dev, stream);
}

template <int G>
cudaError_t launch_group(const Q4Args& a, const void* x, const DeviceInfo& dev, cudaStream_t stream) {
    if (a.M <= 16) return launch_rows<G, 16>(a, x, dev, stream);
    if (a.M <= 32) return launch_rows<G, 32>(a, x, dev, stream);
    return a.M <= 64 ? launch_rows<G, 64>(a, x, dev, stream) : launch_rows<G, 128>(a, x, dev, stream);
}

constexpr size_t kCounters = size_t(1) << 20;      // the products' counters in front of a workspace stay zero
size_t workspace_bytes_of(int M, int K, bool eight) { return eight && M > kWidenRows ? kCounters + static_cast<size_t>(M) * K * 2 : 0; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

int check_sizes(int M, int K, int N, int group) {
    if (M < 0 || K < 1 || N < 1) return TRELLIS_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return TRELLIS_ERR_UNSUPPORTED;
    if (K % group != 0) return TRELLIS_ERR_SHAPE;
    if (M > 65536 || K > (1 << 20) || N > (1 << 20)) return TRELLIS_ERR_UNSUPPORTED;
    return TRELLIS_OK;
}

}  // namespace

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

extern "C" {

int trellis_gemm_q4_workspace_size(int M, int K, int N, int group, int eight, size_t* bytes) {
    using namespace trellis;
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    const int rc = check_sizes(M, K, N, group);
    if (rc != TRELLIS_OK) return rc;
    *bytes = workspace_bytes_of(M, K, eight != 0);
    return TRELLIS_OK;
}

int trellis_gemm_q4(const void* x, const float* x_scales, const uint32_t* codes, const uint16_t* scales, const uint16_t* biases,
                    int M, int K, int N, int group, uint16_t* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_sizes(M, K, N, group);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(biases, 2) || !aligned(x_scales, 4) || !aligned(out, 2))
        return TRELLIS_ERR_ALIGN;
    if (M == 0) return TRELLIS_OK;
    const bool eight = x_scales != nullptr;
    // all of them are read until the last result is stored
    const size_t out_bytes = static_cast<size_t>(M) * N * 2, group_bytes = static_cast<size_t>(N) * (K / group) * 2;
    if (overlap(x, static_cast<size_t>(M) * K * (eight ? 1 : 2), out, out_bytes) || overlap(codes, static_cast<size_t>(N) * K / 2, out, out_bytes) ||
        overlap(scales, group_bytes, out, out_bytes) || (biases != nullptr && overlap(biases, group_bytes, out, out_bytes)) ||
        (eight && overlap(x_scales, static_cast<size_t>(M) * 4, out, out_bytes)))
        return TRELLIS_ERR_SHAPE;
    const size_t need = workspace_bytes_of(M, K, eight);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return TRELLIS_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return TRELLIS_ERR_ALIGN;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    if (need > 0) {
        uint16_t* x16 = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + kCounters);
        const long long count = static_cast<long long>(M) * (K / 8), ctas = (count + 255) / 256, most = 8ll * dev.num_sms;
        if (launch_programmatic(q4_widen_kernel, static_cast<unsigned>(ctas < most ? ctas : most), 256u, 0, stream,
                                static_cast<const uint8_t*>(x), count, x16) != cudaSuccess)
            return TRELLIS_ERR_CUDA;
        x = x16;
    }
    Q4Args a = {};
    a.codes = codes; a.scales = scales; a.biases = biases; a.x_scales = x_scales; a.out = out;
    a.M = M; a.K = K; a.N = N; a.groups = K / group;
    if (eight && need == 0) a.x8 = static_cast<const uint8_t*>(x);
    const cudaError_t e = group == 32 ? launch_group<32>(a, x, dev, stream)
                          : group == 64 ? launch_group<64>(a, x, dev, stream) : launch_group<128>(a, x, dev, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // extern "C"
