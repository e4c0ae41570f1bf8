// Attention over the paged 8-bit cache for many query rows: prompt chunks and
// longer drafts, on the tensor cores (tcgen05).
//
// The same function as the streaming kernel (kv_attention_stream.cu), whose notes on
// scales, f16 queries and weights and the seldom-moved reference hold here too.  With
// 128 rows to a key head's tile the products are a dense contraction:
//
//   S[row, key] = Q K^T    Q [128, D] and K [64, D] f16 in shared memory, both K-major
//   O[row, d]  += P V      P [128, 64] f16 in tensor memory, V [64, D] f16 in shared
//                          memory as the cache has it (tokens x D: "MN-major" for this
//                          product, so nothing is transposed)
//
// A CTA takes one (sequence, 128 query rows of one key head's group, key head), or a
// part of its tokens where there are too few units for the SMs, and runs three roles:
//
// * 4 conversion warps: warp w loads the codes of tokens 16w .. 16w+15 of each 64-token
//   tile (one block of the cache, so one page and one pair of scales), a tile ahead in
//   registers, and stores them as f16 in the 128-byte-swizzled layout that both
//   products read: row = token, 64 values (128 bytes) a row, 16-byte chunk c of row r at
//   c ^ (r % 8), one such panel for each 64 values of D.
// * 1 thread issues the products.  S is double buffered: S of tile i + 1 is issued
//   before the wait for P of tile i.
// * 4 softmax warps, a row a thread: scores from tensor memory, p' = 2^(x - m), sums in
//   registers, P over the columns that S had.  O is rescaled in tensor memory only when
//   a row's reference moves.
//
// What bounds it: at long contexts the 4 D flops a (row, key) pair, against 16
// exponentials a clock and SM at 1 / (4 D) of that rate: for D = 128 the products of a
// 64-key tile and its 8192 exponentials take about equally long.  Two CTAs an SM
// (D <= 128) let one's softmax run beside the other's products.
//
// Waits are bounded as in gemm_tc_kernel.cu: one that gives up sets the device error
// word and its role leaves; the issuing thread always waits for its last products
// before the tensor memory is released.
#include "kv_attention.cuh"
#include "trellis.h"

namespace trellis {

__device__ unsigned int g_kv_error = 0u;

namespace {

constexpr float kMoveBy = 8.0f;
constexpr int kRows = 128;               // query rows of a unit
constexpr int kKeys = 64;                // cached tokens of a tile
constexpr int kSoftWarps = 4, kConvWarps = 4;
constexpr int kThreads = (kSoftWarps + kConvWarps + 1) * 32;
constexpr int kScaleSlots = 4;           // tiles whose scales are held
constexpr int kMinChunk = 4;             // fewest tiles of a split unit's part

template <int D>
struct Tile {
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kKvBytes = kKeys * D * 2;       // a converted key or value tile
    static constexpr int kPanel = kKeys * 128;           // 64 values of each of its tokens
    static constexpr int kQPanel = kRows * 128;
    static constexpr int kOffK = kQBytes;                // two stages each
    static constexpr int kOffV = kOffK + 2 * kKvBytes;
    static constexpr int kOffScale = kOffV + 2 * kKvBytes;
    static constexpr int kOffBar = kOffScale + kScaleSlots * 4 * 16;
    // barriers
    static constexpr int kQFull = 0, kKFull = 1, kSFull = 3, kVFull = 5, kPvDone = 7, kPFull = 9, kDone = 11;
    static constexpr int kOffTaddr = kOffBar + 12 * 8;
    static constexpr int kSmem = kOffTaddr + 32 + 1024;  // + rounding of the base to 1 KB
    static constexpr int kSCol = 0;                      // S / P: 2 x 64 columns
    static constexpr int kOCol = 2 * kKeys;              // O: D columns
    static constexpr int kCols = 2 * kKeys + D <= 256 ? 256 : 512;
    static constexpr int kCtas = D <= 128 ? 2 : 1;       // an SM
    // f16 operands, fp32 sums; N in bits 17-22, M in 24-28; bit 16: B is MN-major
    static constexpr uint32_t kIdescS = (1u << 4) | (static_cast<uint32_t>(kKeys >> 3) << 17) |
                                        (static_cast<uint32_t>(kRows >> 4) << 24);
    static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) |
                                        (static_cast<uint32_t>(kRows >> 4) << 24);
    static constexpr size_t kPart = static_cast<size_t>(kRows) * D + 2 * kRows;   // floats of a part's result
    static_assert(kSmem * kCtas <= 232448, "shared memory");
};

// ---- PTX wrappers ------------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
// Bounded wait: gives up after 2 s of wall-clock time (or 2^26 polls).
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity) {
    unsigned long long t0, t1;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t i = 0; i < (1u << 26); ++i) {
        uint32_t ok;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok != 0u) return true;
        if ((i & 63u) == 63u) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
            if (t1 - t0 > 2000000000ull) break;
        }
    }
    atomicOr(&g_kv_error, 1u);
    return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0u || bar_wait_slow(bar, parity);
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Shared-memory descriptor, 128-byte swizzle: start, leading and stride byte offsets.
// K-major (both operands of S): 1 KB between groups of 8 rows.  MN-major (V): the
// stride offset separates groups of 8 tokens, the leading offset panels of 64 values.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                 "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
                 "%30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                 "%12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                 "%12, %13, %14, %15, %16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                   "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                   "r"(r[15]) : "memory");
}

struct Part {
    int seq, head, qt;
    int start, n, p0, total;
    int lo, hi;              // cached tokens that the unit's rows see, lo a multiple of 64
    int t0, t1;              // its tiles [t0, t1)
    int parts;               // of the unit
};

// The unit and part of work item `item`; false when there is none.  Units are counted
// from the last query tile of the last sequence, so that the long ones of a causal
// prompt come first.  One warp calls it.
__device__ bool find_part(const AttendArgs& a, long long item, int splits, Part& u) {
    const int lane = threadIdx.x & 31;
    const int split = static_cast<int>(item % splits);
    item /= splits;
    u.head = static_cast<int>(item % a.l.kv_heads);
    long long tile = item / a.l.kv_heads;
    int got = -1, qt = 0;
    for (int s1 = a.l.seqs; s1 > 0 && got < 0; s1 -= 32) {
        const int s = s1 - 1 - lane;
        Seq q = {};
        if (s >= 0) q = load_seq(a.l, s);
        const int qts = q.n > 0 ? (q.n * a.group + kRows - 1) / kRows : 0;
        int incl = qts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, tile >= incl - qts && tile < incl);
        if (hit != 0u) {
            const int src = __ffs(hit) - 1;
            qt = __shfl_sync(0xffffffffu, qts - 1 - static_cast<int>(tile - (incl - qts)), src);
            got = s1 - 1 - src;
            u.start = __shfl_sync(0xffffffffu, q.start, src);
            u.n = __shfl_sync(0xffffffffu, q.n, src);
            u.p0 = __shfl_sync(0xffffffffu, q.p0, src);
            u.total = __shfl_sync(0xffffffffu, q.total, src);
        }
        tile -= __shfl_sync(0xffffffffu, incl, 31);
    }
    if (got < 0) return false;
    u.seq = got;
    u.qt = qt;
    const int first = qt * kRows / a.group, last = min(u.n - 1, (qt * kRows + kRows - 1) / a.group);
    u.hi = max(0, min(u.total, u.p0 + last + 1));
    const int low = a.window > 0 ? max(0, u.p0 + first + 1 - a.window) : 0;
    u.lo = low & ~(kKeys - 1);
    const int tiles = u.hi > u.lo ? (u.hi - u.lo + kKeys - 1) / kKeys : 0;
    const int chunk = max(kMinChunk, (tiles + splits - 1) / splits);
    u.parts = max(1, (tiles + chunk - 1) / chunk);
    u.t0 = split * chunk;
    u.t1 = min(tiles, u.t0 + chunk);
    return split < u.parts;
}

template <int D>
__global__ void __launch_bounds__(kThreads, Tile<D>::kCtas)
kv_tile_kernel(const __grid_constant__ AttendArgs a, int splits) {
    using T = Tile<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Part shared_part;
    __shared__ int shared_ok;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    unsigned char* const smem = smem_raw + (sbase - sraw);
    const uint32_t bars = sbase + T::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };

    griddep_wait();
    if (warp == 0) {
        Part p;
        const bool ok = find_part(a, blockIdx.x, splits, p);
        if (lane == 0) { shared_part = p; shared_ok = ok; }
    } else if (threadIdx.x == 32) {
        bar_init(bar(T::kQFull), kSoftWarps);
        for (int s = 0; s < 2; ++s) {
            bar_init(bar(T::kKFull + s), kConvWarps);
            bar_init(bar(T::kSFull + s), 1);
            bar_init(bar(T::kVFull + s), kConvWarps);
            bar_init(bar(T::kPvDone + s), 1);
            bar_init(bar(T::kPFull + s), kSoftWarps);
        }
        bar_init(bar(T::kDone), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    __syncthreads();
    if (!shared_ok) { griddep_launch_dependents(); return; }
    const Part u = shared_part;
    const int tiles = u.t1 - u.t0;                       // 0: the rows see nothing
    if (warp == kSoftWarps + kConvWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(sbase + T::kOffTaddr), "r"(T::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + T::kOffTaddr);
    float4* const scales = reinterpret_cast<float4*>(smem + T::kOffScale);   // [slot][block]: k scale, log2 v, 1 / v

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------------ softmax
        const int r = u.qt * kRows + static_cast<int>(threadIdx.x);
        const int tok = r / a.group;
        const bool live = tok < u.n;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        // this row's query: f16 times a power of two, into the swizzled K-major tile
        float qmul;
        {
            const uint16_t* row = a.q + static_cast<size_t>(u.start + (live ? tok : 0)) * a.q_stride +
                                  (static_cast<size_t>(u.head) * a.group + r % a.group) * D;
            const uint4* r4 = reinterpret_cast<const uint4*>(row);
            uint32_t most = 0u;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = __ldg(r4 + c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) most = max(most, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
            }
            const int e = query_exponent(most);
            const float down = live ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
            qmul = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
            const uint32_t dst = sbase + threadIdx.x * 128;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = __ldg(r4 + c);
                const uint32_t at = dst + (c >> 3) * T::kQPanel + ((static_cast<uint32_t>(c & 7) ^ (threadIdx.x & 7)) << 4);
                sts128(at, f32_to_f16x2(bf16_lo(v.x) * down, bf16_hi(v.x) * down),
                       f32_to_f16x2(bf16_lo(v.y) * down, bf16_hi(v.y) * down),
                       f32_to_f16x2(bf16_lo(v.z) * down, bf16_hi(v.z) * down),
                       f32_to_f16x2(bf16_lo(v.w) * down, bf16_hi(v.w) * down));
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kQFull));
        }
        const int limit = min(u.hi, u.p0 + tok + 1);
        const int lower = a.window > 0 ? u.p0 + tok + 1 - a.window : 0;
        // tokens that every row of the unit sees
        const int all_hi = min(u.hi, u.p0 + u.qt * kRows / a.group + 1);
        const int all_lo = a.window > 0 ? u.p0 + min(u.n - 1, (u.qt * kRows + kRows - 1) / a.group) + 1 - a.window : 0;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            const int b = i & 1;
            const uint32_t par = (i >> 1) & 1;
            // the conversion warps stored the scales before they arrived for V; that barrier
            // cannot run ahead of this wait (V of tile i + 2 needs the product with P of tile
            // i), as the one for K could
            ok = bar_wait(bar(T::kSFull + b), par) && bar_wait(bar(T::kVFull + b), par);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            fence_after();
            const uint32_t s_addr = lane_base + T::kSCol + b * kKeys;
            uint32_t s0[32], s1[32];
            tmem_ld32(s0, s_addr);
            tmem_ld32(s1, s_addr + 32);
            float4 sc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[k] = scales[(i % kScaleSlots) * 4 + k];
            wait_ld();
            const int tok0 = u.lo + (u.t0 + i) * kKeys;
            float top = -INFINITY;
            auto score = [&](uint32_t v, int k, int j) {
                float x = fmaf(__uint_as_float(v), sc[k].x * qmul, sc[k].y);
                return x;
            };
            if (tok0 + kKeys > all_hi || tok0 < all_lo) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float x0 = score(s0[j], j >> 4, j), x1 = score(s1[j], 2 + (j >> 4), j);
                    const int k0 = tok0 + j, k1 = k0 + 32;
                    s0[j] = __float_as_uint(k0 < limit && k0 >= lower ? x0 : -INFINITY);
                    s1[j] = __float_as_uint(k1 < limit && k1 >= lower ? x1 : -INFINITY);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    s0[j] = __float_as_uint(score(s0[j], j >> 4, j));
                    s1[j] = __float_as_uint(score(s1[j], 2 + (j >> 4), j));
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(__uint_as_float(s0[j]), __uint_as_float(s1[j])));
            if (__any_sync(0xffffffffu, top > m + kMoveBy)) {
                const float to = fmaxf(m, top);
                const float f = m == -INFINITY ? 0.0f : exp2_approx(m - to);
                m = to;
                l *= f;
                if (i > 0) {
                    // O holds the tiles before this one
                    ok = bar_wait(bar(T::kPvDone + (b ^ 1)), ((i - 1) >> 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o, lane_base + T::kOCol + c);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st16(lane_base + T::kOCol + c, o);
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float part = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p0 = exp2_approx(__uint_as_float(s0[16 * k + 2 * j]) - ref);
                    const float p1 = exp2_approx(__uint_as_float(s0[16 * k + 2 * j + 1]) - ref);
                    part += p0 + p1;
                    p[8 * k + j] = f32_to_f16x2(p0, p1);
                }
                l = fmaf(part, sc[k].z, l);
            }
            tmem_st16(s_addr, p);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float part = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p0 = exp2_approx(__uint_as_float(s1[16 * k + 2 * j]) - ref);
                    const float p1 = exp2_approx(__uint_as_float(s1[16 * k + 2 * j + 1]) - ref);
                    part += p0 + p1;
                    p[8 * k + j] = f32_to_f16x2(p0, p1);
                }
                l = fmaf(part, sc[2 + k].z, l);
            }
            tmem_st16(s_addr + 16, p);
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kPFull + b));
        }
        // ---- result -------------------------------------------------------------------
        if (ok && tiles > 0) {
            ok = bar_wait(bar(T::kPvDone + ((tiles - 1) & 1)), ((tiles - 1) >> 1) & 1);
            fence_after();
        }
        ok = __all_sync(0xffffffffu, ok);
        const bool whole = u.parts == 1;
        const long long unit = blockIdx.x / splits;
        float* part = whole ? nullptr : a.partials + (unit * splits + blockIdx.x % splits) * T::kPart;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = a.out + ((static_cast<size_t>(u.start) + (live ? tok : 0)) * a.l.q_heads +
                                 static_cast<size_t>(u.head) * a.group + r % a.group) * D;
        if (ok) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                if (tiles > 0) {
                    tmem_ld16(o, lane_base + T::kOCol + c);
                    wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0u;
                }
                if (whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        // a row that sees nothing is zero, whatever its sums are
                        w[j] = l == 0.0f ? 0u : pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    if (live) {
                        reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * kRows + threadIdx.x] = __uint_as_float(o[j]);
                }
            }
            if (!whole) {
                part[D * kRows + threadIdx.x] = m;
                part[D * kRows + kRows + threadIdx.x] = l;
                // the part that finishes last adds them all, in their order
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (threadIdx.x == 0) {
                    const unsigned int got = atomicAdd(a.counters + unit, 1u);
                    shared_ok = got == static_cast<unsigned int>(u.parts - 1);
                    if (shared_ok) a.counters[unit] = 0u;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (shared_ok && live) {
                    __threadfence();
                    const float* base = a.partials + unit * splits * T::kPart + threadIdx.x;
                    float top = -INFINITY;
                    for (int q = 0; q < u.parts; ++q) top = fmaxf(top, __ldcg(base + q * T::kPart + D * kRows));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    float den = 0.0f;
                    for (int q = 0; q < u.parts; ++q) {
                        const float* p = base + q * T::kPart + D * kRows;
                        den = fmaf(__ldcg(p + kRows), exp2_approx(__ldcg(p) - ref), den);
                    }
                    const float s = 1.0f / den;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float acc[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
                        for (int q = 0; q < u.parts; ++q) {
                            const float* p = base + q * T::kPart;
                            const float f = exp2_approx(__ldcg(p + D * kRows) - ref);
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[j] = fmaf(__ldcg(p + (c + j) * kRows), f, acc[j]);
                        }
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = den == 0.0f ? 0u : pack_bf16x2(acc[2 * j] * s, acc[2 * j + 1] * s);
                        reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
            }
        }
    } else if (warp < kSoftWarps + kConvWarps) {
        // --------------------------------------------------------------- conversion
        constexpr int P = D / 64;                        // panels of 64 values
        const int w = warp - kSoftWarps;                 // tokens 16w .. 16w + 15 of a tile
        const int c4 = lane & 3, r8 = lane >> 2;         // 16 codes c4 of a panel's 64, tokens r8 and r8 + 8
        uint4 kraw[2][P], vraw[2][P];
        float ks = 0.0f, vs = 0.0f;
        // codes of tile i: base of this warp's block (null past the last token)
        auto block_of = [&](int i, size_t* unit, int* in_page) {
            const int t = u.lo + (u.t0 + i) * kKeys + 16 * w;
            if (t >= u.hi) return false;
            *unit = static_cast<size_t>(kv_page(a.l, u.seq, t >> a.l.page_shift)) * a.l.kv_heads + u.head;
            *in_page = t & (a.l.page_size - 1);
            return true;
        };
        auto load = [&](const uint8_t* codes, size_t unit, int in_page, bool in, uint4 (&raw)[2][P]) {
            const uint8_t* src = codes + (unit * a.l.page_size + in_page) * D + c4 * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    raw[h][p] = in ? __ldg(reinterpret_cast<const uint4*>(src + (r8 + 8 * h) * D + p * 64))
                                   : make_uint4(0u, 0u, 0u, 0u);
        };
        // store as f16: token row 16w + 8h + r8 of panel p, chunks 2 c4 and 2 c4 + 1
        auto store = [&](uint32_t dst, const uint4 (&raw)[2][P], int valid) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool keep = r8 + 8 * h < valid;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const uint32_t in[4] = {raw[h][p].x, raw[h][p].y, raw[h][p].z, raw[h][p].w};
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e4m3x4_to_f16x2(keep ? in[j] : 0u, o[2 * j], o[2 * j + 1]);
                    const uint32_t row = dst + p * T::kPanel + (16 * w + 8 * h + r8) * 128;
                    const uint32_t c = 2 * c4;
                    sts128(row + (((c) ^ r8) << 4), o[0], o[1], o[2], o[3]);
                    sts128(row + (((c + 1) ^ r8) << 4), o[4], o[5], o[6], o[7]);
                }
            }
        };
        size_t unit = 0;
        int in_page = 0;
        bool in = tiles > 0 && block_of(0, &unit, &in_page);
        auto load_scales = [&]() {
            const size_t at = unit * (a.l.page_size / kKvBlock) + in_page / kKvBlock;
            ks = in ? __ldg(a.k_scales + at) : 1.0f;
            vs = in ? __ldg(a.v_scales + at) : 1.0f;
        };
        load(a.k_codes, unit, in_page, in, kraw);
        load(a.v_codes, unit, in_page, in, vraw);
        load_scales();
        for (int i = 0; i < tiles; ++i) {
            const int b = i & 1;
            const int valid = u.hi - (u.lo + (u.t0 + i) * kKeys + 16 * w);   // tokens of the block that count
            // stage b is free when the products of tile i - 2 are done
            bool ok = i < 2 || bar_wait(bar(T::kSFull + b), ((i - 2) >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) scales[(i % kScaleSlots) * 4 + w] = make_float4(ks, pow2_log2(vs), pow2_recip(vs), 0.0f);
            store(sbase + T::kOffK + b * T::kKvBytes, kraw, valid);
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kKFull + b));
            const bool more = i + 1 < tiles;
            in = more && block_of(i + 1, &unit, &in_page);
            load(a.k_codes, unit, in_page, in, kraw);
            load_scales();
            ok = i < 2 || bar_wait(bar(T::kPvDone + b), ((i - 2) >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            store(sbase + T::kOffV + b * T::kKvBytes, vraw, valid);
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kVFull + b));
            load(a.v_codes, unit, in_page, in, vraw);
        }
    } else if (lane == 0) {
        // ----------------------------------------------------------------- products
        bool ok = tiles == 0 || bar_wait(bar(T::kQFull), 0);
        auto scores = [&](int i) {
            const uint32_t kb = sbase + T::kOffK + (i & 1) * T::kKvBytes;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k & 3) * 32;       // 16 values inside a panel's 128-byte row
                mma_ss(tmem + T::kSCol + (i & 1) * kKeys, desc(sbase + (k >> 2) * T::kQPanel + off, 16),
                       desc(kb + (k >> 2) * T::kPanel + off, 16), T::kIdescS, k > 0);
            }
            commit(bar(T::kSFull + (i & 1)));
        };
        if (ok && tiles > 0) {
            ok = bar_wait(bar(T::kKFull), 0);
            if (ok) { fence_after(); scores(0); }
        }
        for (int i = 0; i < tiles && ok; ++i) {
            const int b = i & 1;
            const uint32_t par = (i >> 1) & 1;
            if (i + 1 < tiles) {
                // S of tile i + 1 takes the columns that P of tile i - 1 had: its product
                // was issued before by this thread, and the tensor pipe runs in order
                ok = bar_wait(bar(T::kKFull + (b ^ 1)), ((i + 1) >> 1) & 1);
                if (!ok) break;
                fence_after();
                scores(i + 1);
            }
            ok = bar_wait(bar(T::kVFull + b), par) && bar_wait(bar(T::kPFull + b), par);
            if (!ok) break;
            fence_after();
            const uint32_t vb = sbase + T::kOffV + b * T::kKvBytes;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
                mma_ts(tmem + T::kOCol, tmem + T::kSCol + b * kKeys + k * 8, desc(vb + k * 2048, T::kPanel), T::kIdescO,
                       i > 0 || k > 0);
            commit(bar(T::kPvDone + b));
        }
        // nothing is in flight when the tensor memory is released
        commit(bar(T::kDone));
        (void)bar_wait(bar(T::kDone), 0);
    }

    griddep_launch_dependents();
    fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kConvWarps) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(T::kCols) : "memory");
    }
}

// Units that the packed rows can make (their lengths are on the device): a partial tile
// a sequence at most.
long long unit_bound(int tokens, int seqs, int group, int kv_heads) {
    const long long rows = static_cast<long long>(tokens) * group;
    const long long t = rows / kRows + seqs, most = rows;
    return (t < most ? t : most) * kv_heads;
}

// Parts that a unit's tokens are cut into: one where the units fill the SMs' CTAs
// twice, else enough for that.
int split_count(long long units, int ctas) {
    const long long want = 2ll * ctas;
    if (units >= want) return 1;
    const long long s = (want + units - 1) / units;
    return static_cast<int>(s);
}

template <int D>
int launch(const AttendArgs& a, long long units, int splits, cudaStream_t stream) {
    using T = Tile<D>;
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(kv_tile_kernel<D>, T::kSmem, opted)) return TRELLIS_ERR_CUDA;
    const cudaError_t e = launch_programmatic(kv_tile_kernel<D>, static_cast<unsigned>(units * splits),
                                              static_cast<unsigned>(kThreads), T::kSmem, stream, a, splits);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // namespace

size_t kv_tile_workspace_bytes(int tokens, int seqs, int q_heads, int kv_heads, int head_dim, const DeviceInfo& dev) {
    const long long units = unit_bound(tokens > 0 ? tokens : 1, seqs, q_heads / kv_heads, kv_heads);
    const int splits = split_count(units, dev.num_sms * (head_dim <= 128 ? 2 : 1));
    if (splits == 1) return kKvCounterBytes;
    return kKvCounterBytes + static_cast<size_t>(units) * splits * (static_cast<size_t>(kRows) * head_dim + 2 * kRows) * 4;
}

int launch_kv_tile(const AttendArgs& a, int head_dim, const DeviceInfo& dev, cudaStream_t stream) {
    const long long units = unit_bound(a.l.tokens, a.l.seqs, a.group, a.l.kv_heads);
    const int splits = split_count(units, dev.num_sms * (head_dim <= 128 ? 2 : 1));
    if (units * splits >= (1ll << 31)) return TRELLIS_ERR_SHAPE;
    return head_dim == 64 ? launch<64>(a, units, splits, stream)
           : head_dim == 128 ? launch<128>(a, units, splits, stream) : launch<256>(a, units, splits, stream);
}

int kv_take_device_error(unsigned int* flags) {
    unsigned int v = 0u;
    if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v)) != cudaSuccess) return -5;
    if (v != 0u) {
        const unsigned int zero = 0u;
        if (cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero)) != cudaSuccess) return -5;
    }
    *flags = v;
    return 0;
}

}  // namespace trellis
