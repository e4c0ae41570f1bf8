// Attention over the paged 8-bit cache for many query rows: prompt chunks and
// longer drafts, on the tensor cores (tcgen05).
//
// The same function as the streaming kernel (kv_attention_stream.cu), whose notes on
// scales and on the seldom-moved reference hold here too.  With 128 rows to a key head's
// tile the products are a dense contraction:
//
//   S[row, key] = Q K^T    K: the cache's e4m3 codes as they are, [64 keys, D] in shared
//                          memory.  A bf16 query has 8 significant bits and e4m3 4, so
//                          q = hi + lo in two e4m3 numbers, the row being scaled by a
//                          power of two: exactly down to 2^-9 of the row's largest
//                          value, within 2^-17 of that value below.  Two 8-bit products
//                          at twice the rate of one 16-bit product, and keys need no
//                          conversion.
//   O[row, d]  += P V      P [128, 64] f16 in tensor memory over the columns that S had,
//                          V converted to f16 in shared memory as the cache has it
//                          (tokens x D: "MN-major" for this product, nothing is transposed).
//                          Weights need more than e4m3's bits; f16 keeps 11.
//
// A CTA an SM works through items: (sequence, QT x 128 query rows of one key head's
// group, key head), or where there are too few units for the SMs an equal share of all
// units' tiles, cut where it falls (kv_join_kernel adds the parts up).
// QT = 2 query tiles share every loaded tile of keys and values (1 at D = 256, whose sums
// fill tensor memory), and one's softmax runs beside the other's products.  Roles:
//
// * 1 warp plans: finds the next item's rows, shortly before the one at hand ends.
// * 4 warps load (8 at D = 256): warp w the codes of tokens 16w .. 16w+15 of each 64-token
//   tile (one block of the cache, so one page and one pair of scales; half of one at D = 256),
//   a tile ahead in registers, keys one further; K goes to shared memory as it is, V as f16,
//   both in the 128-byte-swizzled layout: row = token, 128 bytes a row (a panel), 16-byte
//   chunk c of row r at c ^ (r % 8).
// * 1 warp issues the products.
// * 4 warps a query tile do the softmax, a row a thread: scores from tensor memory,
//   p' = 2^(x - m), sums in registers.  O is rescaled in tensor memory only when a row's
//   reference moves.  They also store the result and bring in the next item's queries.
//
// What bounds it: per 64-key tile and 128 rows at D = 128 the products take 512 clocks of the
// tensor pipe; but a row's softmax is one thread's chain of some 1000
// to 1400 clocks (scores out of tensor memory, maximum, exponentials, P back), two warps a
// scheduler, and an item costs 10 to 14 thousand clocks of its own (queries, first and last
// products, result).  Measured (GPU time; the least bytes or operations at 6.69 TB/s and
// 1951 TFLOP/s): chunks of 4 x 2048 tokens on contexts of 4100 to 9001, 32 / 8 heads of 128:
// 672 us (351), 1.02 PFLOP/s; 6 prompts of 130 to 4099 tokens, window 1024, 24 / 8 heads of 64:
// 157 us (31), where a row-tile has half of the products to the same softmax; 16 x 5 drafts on
// contexts of 300 to 9000, 32 / 4 heads of 256: 70 us (23), one query tile of 40 rows, so that
// nothing runs beside its chain.
//
// Waits are bounded as in gemm_tc_kernel.cu: one that gives up sets the device error
// word and its role leaves; the issuing warp always waits for its last products
// before the tensor memory is released.
#include "kv_attention.cuh"
#include "trellis.h"

namespace trellis {

__device__ unsigned int g_kv_error = 0u;

namespace {

// The reference moves when exceeded by 2^15.9: weights are at most that (f16 ends at 65504), and the
// move, a pass over O of some 1500 to 3800 clocks, is rare (at 2^8 the chunks above took 702 us
// for 664, the windowed prompts 166 for 157).  It moves to the largest score over 2^below, because
// weights under 2^-25 vanish in f16 but count in the denominators: N tokens then lose at most
// N 2^-(25 + below) of the largest weight, and below = log2(N) - kNear, rounded up, keeps that
// under 2^-14 up to 2^21 tokens.  Units of up to 2^11 tokens need none.  (Chunks 663 us without it,
// 670 to 672 so; 677, 683, 690, 699 with 4 to 7 at every length.)
constexpr float kMoveBy = 15.9f;
constexpr int kNear = 11, kFarBelow = 10;
constexpr int kRows = 128;               // query rows of a tile (lanes of tensor memory)
constexpr int kKeys = 64;                // cached tokens of a tile
constexpr int kScaleSlots = 8;           // tiles whose scales are held
constexpr int kFar = 4;                  // tiles ahead that are brought to L2
constexpr int kMinChunk = 4;             // fewest tiles of a split unit's part

template <int D>
struct Tile {
    static constexpr int kQt = D <= 128 ? 2 : 1;         // query tiles of a CTA
    static constexpr int kSoftWarps = 4 * kQt;
    // loading warps: 16 tokens of a tile each, or 8 where the one query tile leaves room for more warps
    static constexpr int kLoadWarps = D == 256 ? 8 : 4;
    static constexpr int kLoadToks = kKeys / kLoadWarps;
    static constexpr int kThreads = (kSoftWarps + kLoadWarps + 2) * 32;
    static constexpr int kKStages = 2, kVStages = 3;     // tiles of keys and of values in shared memory
    static constexpr int kPanel = kKeys * 128;           // 128 bytes of each token of a tile
    static constexpr int kKPanels = D <= 128 ? 1 : 2;    // a D = 64 row takes half of its 128 bytes
    static constexpr int kVPanels = D / 64;
    // queries: hi and lo terms of 128 bytes a row and panel; at D = 64 one row holds both
    static constexpr int kQPanel = kRows * 128;
    static constexpr int kQTerm = kKPanels * kQPanel;    // from a row's hi term to its lo term (64 bytes at D = 64)
    static constexpr int kQBytes = D == 64 ? kQPanel : 2 * kQTerm;
    static constexpr int kOffK = kQt * kQBytes;
    static constexpr int kOffV = kOffK + kKStages * kKPanels * kPanel;
    static constexpr int kOffStage = kOffV + kVStages * kVPanels * kPanel;   // results on their way out: 32 rows a warp
    static constexpr int kStageD = D == 128 ? 128 : 64;                     // values of a row at a time
    static constexpr int kStageWarp = 32 * kStageD * 2;
    static constexpr int kOffScale = kOffStage + kSoftWarps * kStageWarp;
    static constexpr int kOffMul = kOffScale + kScaleSlots * 4 * 16;         // a float a query row
    static constexpr int kOffPart = kOffMul + kQt * kRows * 4;
    static constexpr int kOffBar = kOffPart + 2 * 64;
    // barriers
    static constexpr int kQFull = 0, kKFull = kQt, kVFull = kKFull + kKStages, kSFull = kVFull + kVStages,
                         kPFull = kSFull + 2 * kQt, kItem = kPFull + 2 * kQt, kPartFull = kItem + kQt, kPartFree = kPartFull + 2,
                         kDone = kPartFree + 2, kBars = kDone + 1;
    static constexpr int kOffTaddr = kOffBar + kBars * 8;
    static constexpr int kSmem = kOffTaddr + 32 + 1024;  // + rounding of the base to 1 KB
    // tensor memory: two tiles of scores (P over them) and the sums of each query tile
    static constexpr int kSCol = 0;
    static constexpr int kOCol = kSCol + kQt * 2 * kKeys;
    static constexpr int kCols = 512;
    // fp32 sums; N in bits 17-22, M in 24-28; formats 0 are e4m3 and f16; bit 16: B is MN-major
    static constexpr uint32_t kIdescS = (1u << 4) | (static_cast<uint32_t>(kKeys >> 3) << 17) |
                                        (static_cast<uint32_t>(kRows >> 4) << 24);
    static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) |
                                        (static_cast<uint32_t>(kRows >> 4) << 24);
    static constexpr size_t kPart = static_cast<size_t>(kRows) * D + 2 * kRows;   // floats of a query tile's partial result
    static_assert(kOCol + kQt * D <= kCols, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ uint4 ldg_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
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
// The products' instructions below are executed by the elected lane of a warp whose
// lanes all walk the same path: their operands then live in uniform registers, which a
// branch of one lane would have to fill one by one before every product.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t elected) {
    asm volatile("{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
                 :: "r"(bar), "r"(elected) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Shared-memory descriptor, 128-byte swizzle: start, leading and stride byte offsets.
// K-major (keys): 1 KB between groups of 8 tokens.  MN-major (values): the stride offset
// separates groups of 8 tokens, the leading offset panels of 64 values.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// One 8-bit product (K = 32) with both operands in shared memory, and one f16 product
// (K = 16) with A in tensor memory.  The issuing warp is the bottleneck if an issue costs
// it more than the product (48 and 64 clocks here), so descriptors are a base and an
// immediate: offsets (in 16 bytes) only reach the address field.
template <int kOffA, int kOffB, bool kAcc>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t elected) {
    asm volatile("{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %7, 0;\n"
                 " add.s64 x, %1, %5;\n add.s64 y, %2, %6;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "n"(kAcc ? 1 : 0), "n"(kOffA >> 4), "n"(kOffB >> 4), "r"(elected)
                 : "memory");
}
template <int kOffA, int kOffB>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t elected) {
    asm volatile("{\n .reg .pred p, e;\n .reg .b64 y;\n .reg .b32 x;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %7, 0;\n"
                 " add.s32 x, %1, %5;\n add.s64 y, %2, %6;\n"
                 " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "n"(kOffA), "n"(kOffB >> 4), "r"(elected) : "memory");
}
// A tile's products, unrolled.
template <int D, int kTerm, int kStep>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t elected) {
    using T = Tile<D>;
    constexpr int off = (kStep >> 2) * T::kQPanel + (kStep & 3) * 32;
    mma_e4m3<off + kTerm * (D == 64 ? 64 : T::kQTerm), (kStep >> 2) * T::kPanel + (kStep & 3) * 32, (kTerm + kStep > 0)>(
        d, q, k, T::kIdescS, elected);
    if constexpr (kStep + 1 < D / 32) mma_scores<D, kTerm, kStep + 1>(d, q, k, elected);
    else if constexpr (kTerm == 0) mma_scores<D, 1, 0>(d, q, k, elected);
}
template <int D, int kStep>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t p, uint64_t v, uint32_t acc, uint32_t elected) {
    mma_f16<kStep * 8, kStep * 2048>(d, p, v, Tile<D>::kIdescO, acc, elected);
    if constexpr (kStep + 1 < kKeys / 16) mma_values<D, kStep + 1>(d, p, v, 1u, elected);
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

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" :: "r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Part {
    int seq, head, qt;       // qt: in units of kQt query tiles
    int start, n, p0;
    int lo, hi;              // cached tokens that the unit's rows see, lo a multiple of 64
    int t0, t1;              // its tiles [t0, t1)
    int live;                // query tiles that have rows; 0: no more items
    int slot;                // of its partial result; -1: it is all of its unit
};
static_assert(sizeof(Part) <= 64, "part slot");

// Tiles of query tile group `qt` of a sequence, and the tokens [lo, hi) that its rows see.
template <int kUnitRows>
__device__ __forceinline__ int unit_tiles(const AttendArgs& a, const Seq& q, int qt, int* lo, int* hi) {
    const int first = qt * kUnitRows / a.group, last = min(q.n - 1, (qt * kUnitRows + kUnitRows - 1) / a.group);
    *hi = max(0, min(q.total, q.p0 + last + 1));
    const int low = a.window > 0 ? max(0, q.p0 + first + 1 - a.window) : 0;
    *lo = low & ~(kKeys - 1);
    return *hi > *lo ? (*hi - *lo + kKeys - 1) / kKeys : 0;
}
template <int kUnitRows>
__device__ __forceinline__ int unit_count(const AttendArgs& a, const Seq& q) {   // of a sequence and head
    return q.n > 0 ? (q.n * a.group + kUnitRows - 1) / kUnitRows : 0;
}
template <int kUnitRows>
__device__ __forceinline__ int fill_part(const AttendArgs& a, const Seq& q, int seq, int head, int qt, Part& u) {
    u.seq = seq; u.head = head; u.qt = qt;
    u.start = q.start; u.n = q.n; u.p0 = q.p0;
    u.live = min(kUnitRows, q.n * a.group - qt * kUnitRows + kRows - 1) / kRows;
    u.slot = -1;
    return unit_tiles<kUnitRows>(a, q, qt, &u.lo, &u.hi);
}
__device__ __forceinline__ Seq seq_of_lane(const Seq& q, int src) {
    Seq r;
    r.start = __shfl_sync(0xffffffffu, q.start, src);
    r.n = __shfl_sync(0xffffffffu, q.n, src);
    r.p0 = __shfl_sync(0xffffffffu, q.p0, src);
    r.total = __shfl_sync(0xffffffffu, q.total, src);
    return r;
}

// Many units: item `item` is a whole one; false past the last.  They are counted from the
// last query tiles of the last sequence, so that the long ones of a causal prompt come
// first.  One warp calls it.
template <int kUnitRows>
__device__ bool find_unit(const AttendArgs& a, unsigned int item, Part& u) {
    const int lane = threadIdx.x & 31;
    int at = static_cast<int>(item / a.l.kv_heads);
    for (int s1 = a.l.seqs; s1 > 0; s1 -= 32) {
        const int s = s1 - 1 - lane;
        Seq q = {};
        if (s >= 0) q = load_seq(a.l, s);
        const int qts = unit_count<kUnitRows>(a, q);
        int incl = qts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at >= incl - qts && at < incl);
        if (hit != 0u) {
            const int src = __ffs(hit) - 1;
            const int qt = __shfl_sync(0xffffffffu, qts - 1 - (at - (incl - qts)), src);
            u.t0 = 0;
            u.t1 = fill_part<kUnitRows>(a, seq_of_lane(q, src), s1 - 1 - src, static_cast<int>(item % a.l.kv_heads), qt, u);
            return true;
        }
        at -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// Few units: their tiles in a row, and kLead places before each unit's for what an item
// costs a CTA beside its tiles (its queries, its result), are cut into equal shares, one a
// CTA.  So a CTA holds at most one part that began before it and one that goes on
// after it: its two slots of partial results.  Where the longest unit has few tiles the
// units are taken whole instead: of 40-row drafts at D = 128 with contexts of 5 to 100 per
// cent of the most, 320 units of up to 600 tokens take 53 us in shares and 37 whole, up to
// 2000 tokens (32 tiles) 68 and 67, up to 4500 105 and 126, up to 12000 217 and 301.
constexpr int kLead = 10;
constexpr int kWhole = 32;
template <int kUnitRows>
__device__ __forceinline__ int unit_places(const AttendArgs& a, const Seq& q, int qt) {
    int lo, hi;
    return kLead + max(1, unit_tiles<kUnitRows>(a, q, qt, &lo, &hi));    // an empty unit still writes its zeros
}
// Places of a head of each lane's sequence; `longest` is raised to its longest unit's.  The
// warp shares the sequences of many units.
template <int kUnitRows>
__device__ long long head_places(const AttendArgs& a, const Seq& q, int& longest) {
    const int lane = threadIdx.x & 31, qts = unit_count<kUnitRows>(a, q);
    long long sum = 0;
    if (qts <= 4)
        for (int qt = 0; qt < qts; ++qt) {
            const int n = unit_places<kUnitRows>(a, q, qt);
            sum += n;
            longest = max(longest, n);
        }
    for (unsigned many = __ballot_sync(0xffffffffu, qts > 4); many != 0u; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const Seq of = seq_of_lane(q, src);
        const int n = __shfl_sync(0xffffffffu, qts, src);
        long long part = 0;
        for (int qt = lane; qt < n; qt += 32) {
            const int w = unit_places<kUnitRows>(a, of, qt);
            part += w;
            longest = max(longest, w);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == src) sum = part;
    }
    return sum;
}
// Places of a CTA's share, 0: units are taken whole.  One warp calls it, as the next.
template <int kUnitRows>
__device__ long long share_places(const AttendArgs& a, int ctas, long long* all) {
    const int lane = threadIdx.x & 31;
    long long sum = 0;
    int longest = 0;
    for (int s0 = 0; s0 < a.l.seqs; s0 += 32) {
        Seq q = {};
        if (s0 + lane < a.l.seqs) q = load_seq(a.l, s0 + lane);
        sum += head_places<kUnitRows>(a, q, longest);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    *all = sum * a.l.kv_heads;
    if (!__any_sync(0xffffffffu, longest > kLead + kWhole)) return 0;
    return max(static_cast<long long>(kLead + kMinChunk), (*all + ctas - 1) / ctas);
}
// The unit that holds a place (of [0, all)), as a part with all of its tiles, and its first place.
template <int kUnitRows>
__device__ long long find_place(const AttendArgs& a, long long place, Part& u) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    int longest = 0;
    for (int s0 = 0; s0 < a.l.seqs; s0 += 32) {
        Seq q = {};
        if (s0 + lane < a.l.seqs) q = load_seq(a.l, s0 + lane);
        const long long each = head_places<kUnitRows>(a, q, longest), mine = each * a.l.kv_heads;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const long long first = before + incl - mine;
        const unsigned hit = __ballot_sync(0xffffffffu, place >= first && place < first + mine);
        if (hit != 0u) {
            const int src = __ffs(hit) - 1;
            const Seq of = seq_of_lane(q, src);
            const long long per = __shfl_sync(0xffffffffu, each, src);
            long long at = __shfl_sync(0xffffffffu, first, src);
            const int head = static_cast<int>((place - at) / per);
            at += head * per;
            const int qts = unit_count<kUnitRows>(a, of);
            for (int qt0 = 0; qt0 < qts; qt0 += 32) {
                const int w = qt0 + lane < qts ? unit_places<kUnitRows>(a, of, qt0 + lane) : 0;
                int upto = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += up;
                }
                const unsigned in = __ballot_sync(0xffffffffu, place < at + upto);
                if (in != 0u) {
                    const int k = __ffs(in) - 1;
                    at += __shfl_sync(0xffffffffu, upto - w, k);
                    u.t0 = 0;
                    u.t1 = fill_part<kUnitRows>(a, of, s0 + src, head, qt0 + k, u);
                    return at;
                }
                at += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    u.live = 0;
    return 0;
}

template <int D>
__global__ void __launch_bounds__(Tile<D>::kThreads, 1)
kv_tile_kernel(const __grid_constant__ AttendArgs a, bool split, unsigned int items) {
    using T = Tile<D>;
    constexpr int kQt = T::kQt;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sraw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    unsigned char* const smem = smem_raw + (sbase - sraw);
    const uint32_t bars = sbase + T::kOffBar;
    auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
    constexpr int kMmaWarp = T::kSoftWarps + T::kLoadWarps;   // and the planner's after it

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::kKStages; ++s) bar_init(bar(T::kKFull + s), T::kLoadWarps);
        for (int s = 0; s < T::kVStages; ++s) bar_init(bar(T::kVFull + s), T::kLoadWarps);
        for (int q = 0; q < kQt; ++q) {
            bar_init(bar(T::kQFull + q), 4);
            bar_init(bar(T::kSFull + 2 * q), 1);
            bar_init(bar(T::kSFull + 2 * q + 1), 1);
            bar_init(bar(T::kItem + q), 1);
            bar_init(bar(T::kPFull + 2 * q), 4);
            bar_init(bar(T::kPFull + 2 * q + 1), 4);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(bar(T::kPartFull + s), 1);
            bar_init(bar(T::kPartFree + s), T::kSoftWarps + T::kLoadWarps + 1);
        }
        bar_init(bar(T::kDone), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(sbase + T::kOffTaddr), "r"(T::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + T::kOffTaddr), 0);
    float4* const scales = reinterpret_cast<float4*>(smem + T::kOffScale);   // [slot][block]: k scale, log2 v, 1 / v
    griddep_wait();

    // Every role walks the same items: the planner's slot k & 1 holds item k.
    auto part_at = [&](int k) { return reinterpret_cast<volatile Part*>(smem + T::kOffPart + (k & 1) * 64); };
    auto free_part = [&](int k) {
        __syncwarp();
        if (lane == 0) bar_arrive(bar(T::kPartFree + (k & 1)));
    };
    auto take_part = [&](int k, Part& u) {
        if (!bar_wait(bar(T::kPartFull + (k & 1)), (k >> 1) & 1)) return false;
        const volatile int* from = reinterpret_cast<const volatile int*>(part_at(k));
        int* to = reinterpret_cast<int*>(&u);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(Part) / 4); ++i) to[i] = from[i];
        return u.live > 0;
    };

    if (warp < T::kSoftWarps) {
        // ------------------------------------------------------------------ softmax
        const int qi = warp >> 2;                        // query tile
        const int row = static_cast<int>(threadIdx.x) & (kRows - 1);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_base = lane_base + T::kSCol + qi * 2 * kKeys;
        const uint32_t o_addr = lane_base + T::kOCol + qi * D;
        uint32_t turns = 0, tiles_so_far = 0, items = 0; // this query tile's, before this item
        uint32_t vst = 0, vturn = 0, slot = 0;           // value stage and its turn, scale slot, of the next tile
        // The score barriers take turns, one a tile and one more an item (see the products).  Two
        // barriers: a parity tells a turn from the next only, so a wait must never be two turns
        // of a barrier early or late
        auto turn_done = [&](uint32_t n) { return bar_wait(bar(T::kSFull + 2 * qi) + 8 * (n & 1), (n >> 1) & 1); };
        // The queries of an item: its 32 rows of this warp, whole lines at a time, as a power of
        // two times hi + lo in swizzled K-major rows.
        constexpr int kLanes = D / 8;                    // lanes of a row, 8 values each
        const int w0 = (warp & 3) * 32;                  // this warp's first row of the query tile
        float* const muls = reinterpret_cast<float*>(smem + T::kOffMul) + qi * kRows;
        auto load_queries = [&](const Part& v) {
            if (qi >= v.live || v.t1 <= v.t0) return;
            const int c = lane % kLanes, sub = lane / kLanes;
            constexpr int kPer = 32 / kLanes;            // rows of a pass
            const int r0 = (v.qt * kQt + qi) * kRows + w0 + sub;
            constexpr int kSide = kLanes < 16 ? kLanes : 16;
            // (a warp without rows leaves what is there: its rows of S are not looked at)
            if ((v.qt * kQt + qi) * kRows + w0 < v.n * a.group)
#pragma unroll 1
            for (int i0 = 0; i0 < kLanes; i0 += kSide) { // 32 / kPer passes, loaded side by side
                uint4 raw[kSide];
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    const int r = r0 + (i0 + i) * kPer, tok = r / a.group;
                    raw[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (tok < v.n)
                        raw[i] = reinterpret_cast<const uint4*>(
                            a.q + static_cast<size_t>(v.start + tok) * a.q_stride +
                            (static_cast<size_t>(v.head) * a.group + (r - tok * a.group)) * D)[c];
                }
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                    uint32_t most = 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) most = max(most, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                    // the largest lands in [128, 256); a negative score factor turns the query's sign
                    const int e = query_exponent(most);
                    float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * 128.0f;
                    if (a.scale_log2 < 0.0f) down = -down;
                    const int row_in = w0 + (i0 + i) * kPer + sub;
                    // e4m3 has no infinity: a row that holds one, or a NaN, is NaN
                    if (c == 0)
                        muls[row_in] = most >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                            : __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (fabsf(a.scale_log2) * 0.0078125f);
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x0 = bf16_lo(w[2 * h]) * down, x1 = bf16_hi(w[2 * h]) * down;
                        const float x2 = bf16_lo(w[2 * h + 1]) * down, x3 = bf16_hi(w[2 * h + 1]) * down;
                        const uint32_t c01 = f32_to_e4m3x2(x0, x1), c23 = f32_to_e4m3x2(x2, x3);
                        const float2 f01 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(c01)));
                        const float2 f23 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(c23)));
                        hi[h] = c01 | (c23 << 16);
                        lo[h] = static_cast<uint32_t>(f32_to_e4m3x2(x0 - f01.x, x1 - f01.y)) |
                                (static_cast<uint32_t>(f32_to_e4m3x2(x2 - f23.x, x3 - f23.y)) << 16);
                    }
                    // 8 bytes of each term: half of 16-byte chunk c / 2
                    const uint32_t at = sbase + qi * T::kQBytes + (c >> 4) * T::kQPanel + row_in * 128 + (c & 1) * 8;
                    const uint32_t ch = (c >> 1) & 7, r7 = row_in & 7;
                    sts64(at + ((ch ^ r7) << 4), hi[0], hi[1]);
                    if constexpr (D == 64) sts64(at + (((ch + 4) ^ r7) << 4), lo[0], lo[1]);
                    else sts64(at + T::kQTerm + ((ch ^ r7) << 4), lo[0], lo[1]);
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kQFull + qi));
        };
        // Rows of results leave through shared memory, so that stores are whole lines.
        const uint32_t stage = sbase + T::kOffStage + warp * T::kStageWarp;
        auto stage_row = [&](int c, const uint32_t (&w)[8]) {          // values c .. c + 15 of this lane's row
            const uint32_t at = stage + ((c % T::kStageD) >> 6) * 4096 + lane * 128;
            const uint32_t ch = (c >> 3) & 7, r7 = lane & 7;
            sts128(at + ((ch ^ r7) << 4), w[0], w[1], w[2], w[3]);
            sts128(at + (((ch + 1) ^ r7) << 4), w[4], w[5], w[6], w[7]);
        };
        // after the values up to c + 15: stores the last kStageD of the rows when they are complete
        auto store_rows = [&](const Part& v, int c_last) {
            if ((c_last + 16) % T::kStageD != 0) return;
            __syncwarp();
            constexpr int kChunks = T::kStageD / 8;
            const int r0 = (v.qt * kQt + qi) * kRows + w0, c0 = (c_last + 16 - T::kStageD) / 8;
#pragma unroll 4
            for (int i = 0; i < kChunks; ++i) {
                const int at = i * 32 + lane, c = at % kChunks, rr = at / kChunks;
                const int r = r0 + rr, tok = r / a.group;
                const uint4 x = lds128(stage + (c >> 3) * 4096 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
                if (tok < v.n)
                    reinterpret_cast<uint4*>(a.out + ((static_cast<size_t>(v.start) + tok) * a.l.q_heads +
                                                      static_cast<size_t>(v.head) * a.group + (r - tok * a.group)) * D)[c0 + c] = x;
            }
            __syncwarp();
        };
        Part u, next;
        bool have = __all_sync(0xffffffffu, take_part(0, u)), have_next = false;
        free_part(0);
        if (have) load_queries(u);
        for (int k = 0; have; ++k) {
            const bool live_tile = qi < u.live;
            const int r = (u.qt * kQt + qi) * kRows + row;
            const int tok = r / a.group;
            const int tiles = u.t1 - u.t0;               // 0: the rows see nothing
            __syncwarp();
            const float qmul = muls[row];
            const int limit = min(u.hi, u.p0 + tok + 1);
            const int lower = a.window > 0 ? u.p0 + tok + 1 - a.window : 0;
            // tokens that every row of the query tile sees
            const int row0 = (u.qt * kQt + qi) * kRows;
            const int all_hi = min(u.hi, u.p0 + row0 / a.group + 1);
            const int all_lo = a.window > 0 ? u.p0 + min(u.n - 1, (row0 + kRows - 1) / a.group) + 1 - a.window : 0;
            const bool has_rows = row0 + w0 < u.n * a.group;
            // how far the reference stays below the largest score: by the tokens of the unit, not of the part
            const float below = static_cast<float>(min(max(0, 32 - __clz(max(u.hi - u.lo - 1, 0)) - kNear), kFarBelow));
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int i = 0; live_tile && i < tiles; ++i) {
                const uint32_t n = turns + i, pn = tiles_so_far + i;
                // the loaders stored the scales before they arrived for V; that barrier cannot
                // run ahead of this wait (its next use needs the product with this tile's P), as
                // the one for K could
                ok = turn_done(n) && bar_wait(bar(T::kVFull) + 8 * vst, vturn);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                const uint32_t s_addr = s_base + (n & 1) * kKeys;
                uint32_t s0[32], s1[32];
                tmem_ld32(s0, s_addr);
                tmem_ld32(s1, s_addr + 32);
                float mul[4], lv[4], iv[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 v = scales[slot * 4 + c];
                    mul[c] = v.x * qmul; lv[c] = v.y; iv[c] = v.z;
                }
                if (++vst == T::kVStages) { vst = 0; vturn ^= 1; }
                slot = (slot + 1) % kScaleSlots;
                wait_ld();
                if (!has_rows) {                         // P of rows that are not there: whatever it is
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(T::kPFull + 2 * qi) + 8 * (pn & 1));
                    continue;
                }
                const int tok0 = u.lo + (u.t0 + i) * kKeys;
                if (tok0 + kKeys > all_hi || tok0 < all_lo) {
                    // finished scores in the scores' place where some are hidden
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float x0 = fmaf(__uint_as_float(s0[j]), mul[j >> 4], lv[j >> 4]);
                        const float x1 = fmaf(__uint_as_float(s1[j]), mul[2 + (j >> 4)], lv[2 + (j >> 4)]);
                        const int k0 = tok0 + j, k1 = k0 + 32;
                        s0[j] = __float_as_uint(k0 < limit && k0 >= lower ? x0 : -INFINITY);
                        s1[j] = __float_as_uint(k1 < limit && k1 >= lower ? x1 : -INFINITY);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) { mul[c] = 1.0f; lv[c] = 0.0f; }
                }
                // the largest score: scales are positive, so a block's is that of its largest product
                float top = -INFINITY;
                auto block_top = [&](const uint32_t* s, int c) {
                    float x = max3(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
#pragma unroll
                    for (int j = 3; j < 15; j += 2) x = max3(x, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
                    x = fmaxf(x, __uint_as_float(s[15]));
                    top = fmaxf(top, fmaf(x, mul[c], lv[c]));
                };
                block_top(s0, 0); block_top(s0 + 16, 1); block_top(s1, 2); block_top(s1 + 16, 3);
                if (__any_sync(0xffffffffu, top > m + kMoveBy)) {
                    const float to = fmaxf(m, top - below);
                    const float f = m == -INFINITY ? 0.0f : exp2_approx(m - to);
                    m = to;
                    l *= f;
                    if (i > 0) {
                        // O holds the tiles before this one once the next turn is over
                        ok = turn_done(n + 1);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(o, o_addr + c);
                            wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(o_addr + c, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                auto weights = [&](const uint32_t* s, int c, uint32_t* p) {
                    const float2 mm = make_float2(mul[c], mul[c]), sh = make_float2(lv[c] - ref, lv[c] - ref);
                    float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), mm, sh);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        part = __fadd2_rn(part, x);
                        p[j] = f32_to_f16x2(x.x, x.y);
                    }
                    l = fmaf(part.x + part.y, iv[c], l);
                };
                uint32_t p[16];
                weights(s0, 0, p); weights(s0 + 16, 1, p + 8);
                tmem_st16(s_addr, p);
                weights(s1, 2, p); weights(s1 + 16, 3, p + 8);
                tmem_st16(s_addr + 16, p);
                wait_st();
                fence_before();
                __syncwarp();
                // in turn two barriers: a warp may be a tile ahead of the others
                if (lane == 0) bar_arrive(bar(T::kPFull + 2 * qi) + 8 * (pn & 1));
            }
            if (!ok) break;
            if (!live_tile) {                            // the tiles passed by without this query tile
                for (int i = 0; i < tiles; ++i) {
                    if (++vst == T::kVStages) { vst = 0; vturn ^= 1; }
                    slot = (slot + 1) % kScaleSlots;
                }
            }
            if (live_tile && tiles > 0) {                // every S of the item is done: its queries' place is free
                turns += tiles + 1;
                tiles_so_far += tiles;
                if (!__all_sync(0xffffffffu, turn_done(turns - 1))) break;
            }
            // the next item's queries first: its first scores are made while this one's results leave
            have_next = __all_sync(0xffffffffu, take_part(k + 1, next));
            free_part(k + 1);
            if (have_next) load_queries(next);
            // ---- result ---------------------------------------------------------------
            if (live_tile && tiles > 0) {
                ok = bar_wait(bar(T::kItem + qi), items++ & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
            }
            if (live_tile) {
                const bool whole = u.slot < 0;
                float* part = a.partials + (static_cast<size_t>(max(u.slot, 0)) * kQt + qi) * T::kPart;
                const float inv = 1.0f / l;
#pragma unroll 1
                for (int c = 0; has_rows && c < D; c += 16) {
                    uint32_t o[16];
                    if (tiles > 0) {
                        tmem_ld16(o, o_addr + c);
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
                        stage_row(c, w);
                        store_rows(u, c);
                    } else {
                        if (r < u.n * a.group) {
#pragma unroll
                            for (int j = 0; j < 16; j += 4)
                                *reinterpret_cast<uint4*>(part + row * D + c + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                    }
                }
                fence_before();                          // O is read before the next item's products
                if (!whole && r < u.n * a.group) {
                    part[D * kRows + row] = m;
                    part[D * kRows + kRows + row] = l;
                }
            }
            u = next;
            have = have_next;
        }
    } else if (warp < T::kSoftWarps + T::kLoadWarps) {
        // ------------------------------------------------------------------ loads
        constexpr int kToks = T::kLoadToks, kH = kToks / 8;
        const int w = warp - T::kSoftWarps;              // tokens kToks w .. of a tile
        constexpr int kKc = D / 16;                      // 16-byte chunks of a token's codes
        constexpr int kKLoads = kToks * kKc / 32;        // of a lane: whole lines, for K
        constexpr int P = T::kVPanels;
        const int c4 = lane & 3, r8 = lane >> 2;         // for V: 16 codes c4 of a panel's 64, tokens r8 (and r8 + 8)
        // the next tile, on its way in registers (two tiles there measured no faster)
        uint4 kraw[kKLoads], vraw[kH][P];
        float ks = 1.0f, vs = 1.0f;
        Part u = {};
        // stages and scale slot of the next tile; the turns of each query tile's score barriers
        uint32_t kst = 0, vst = 0, slot = 0, turns[kQt];
#pragma unroll
        for (int q = 0; q < kQt; ++q) turns[q] = 0;
        int q_before = -1;                               // last query tile of the item before (-1: none)
        uint32_t turns_before = 0, items[kQt];           // its turns up to that item's end; items of each query tile
#pragma unroll
        for (int q = 0; q < kQt; ++q) items[q] = 0;
        auto turn_done = [&](int q, uint32_t n) { return bar_wait(bar(T::kSFull + 2 * q) + 8 * (n & 1), (n >> 1) & 1); };
        // this warp's block of the tile that is loaded, and the page ids of the next and of a later
        // one, as they were read (they are clamped where they are used: nothing waits before)
        size_t unit = 0;
        int in_page = 0, page_next = 0, page_far = 0;
        auto token_of = [&](int i) { return u.lo + (u.t0 + i) * kKeys + kToks * w; };
        auto seek_page = [&](int i, int tiles) {
            if (i < tiles && token_of(i) < u.hi) page_next = kv_page_id(a.l, u.seq, token_of(i) >> a.l.page_shift);
        };
        auto seek = [&](int i, int tiles) {
            const int t = token_of(i);
            // past the last token: the cache's first block, which nothing looks at (a choice of
            // values instead of addresses would wait for the loads)
            const bool in = i < tiles && t < u.hi;
            unit = in ? static_cast<size_t>(kv_page_of_id(a.l, page_next)) * a.l.kv_heads + u.head : 0;
            in_page = in ? t & (a.l.page_size - 1) : 0;
            seek_page(i + 1, tiles);
            // The registers hold a tile ahead; lines of the tiles after it are brought to L2.
            // (The page id asked for here serves the next call: nothing waits for it.)
            constexpr int kLines = kToks * D / 128;
            const int far = i + kFar, tf = token_of(far);
            if (!split) return;                          // many units: what one reads others have read
            if (i > 0 && far < tiles && tf < u.hi && lane < kLines) {
                const size_t at = ((static_cast<size_t>(kv_page_of_id(a.l, page_far)) * a.l.kv_heads + u.head) * a.l.page_size +
                                   (tf & (a.l.page_size - 1))) * D + lane * 128;
                asm volatile("prefetch.global.L2 [%0];" :: "l"(a.k_codes + at));
                asm volatile("prefetch.global.L2 [%0];" :: "l"(a.v_codes + at));
            }
            if (far + 1 < tiles && token_of(far + 1) < u.hi) page_far = kv_page_id(a.l, u.seq, token_of(far + 1) >> a.l.page_shift);
        };
        auto load_keys = [&](int i, int tiles) {
            seek(i, tiles);
            const uint8_t* src = a.k_codes + (unit * a.l.page_size + in_page) * D + lane * 16;
#pragma unroll
            for (int r = 0; r < kKLoads; ++r) kraw[r] = ldg_once(src + r * 512);
        };
        // the values of the tile that was sought last
        auto load_values = [&] {
            const uint8_t* src = a.v_codes + (unit * a.l.page_size + in_page) * D + c4 * 16;
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int p = 0; p < P; ++p) vraw[h][p] = ldg_once(src + (r8 + 8 * h) * D + p * 64);
            const size_t at = unit * (a.l.page_size / kKvBlock) + in_page / kKvBlock;
            ks = a.k_scales[at];
            vs = a.v_scales[at];
        };
        auto store_keys = [&] {
            const uint32_t kdst = sbase + T::kOffK + kst * T::kKPanels * T::kPanel;
#pragma unroll
            for (int r = 0; r < kKLoads; ++r) {
                const int chunk = r * 32 + lane, tk = chunk / kKc, c = chunk % kKc;
                sts128(kdst + (c >> 3) * T::kPanel + (kToks * w + tk) * 128 + (((c & 7) ^ (tk & 7)) << 4), kraw[r].x, kraw[r].y,
                       kraw[r].z, kraw[r].w);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(T::kKFull) + 8 * kst);
            if (++kst == T::kKStages) kst = 0;
        };
        bool run = true;
        for (int k = 0; run; ++k) {
            if (!__all_sync(0xffffffffu, take_part(k, u))) break;
            const int tiles = u.t1 - u.t0;
            seek_page(0, tiles);
            load_keys(0, tiles);
            load_values();
            const int q_last = u.live - 1;
            uint32_t base = 0;
#pragma unroll
            for (int q = 0; q < kQt; ++q)
                if (q == q_last) base = turns[q];
            auto item_done = [&]() {                     // all products of the item before
                uint32_t n = 0;
#pragma unroll
                for (int q = 0; q < kQt; ++q)
                    if (q == q_before) n = items[q];
                return bar_wait(bar(T::kItem + q_before), (n - 1) & 1);
            };
            if (tiles == 0) free_part(k);
            // Keys go a tile ahead of the values: their product is wanted first.  At an item's
            // start the stages are free when the last turn of the one before is over
            if (tiles > 0) {
                if (!__all_sync(0xffffffffu, q_before < 0 || turn_done(q_before, turns_before - 1))) break;
                store_keys();
                load_keys(1, tiles);
            }
            for (int i = 0; i < tiles; ++i) {
                // the next item is taken when this one nears its end, not before: it may be long
                if (i == max(0, tiles - 4)) free_part(k);
                // turn base + i - 1: S of the tile before is done, and the product with P of the
                // one two before that.  So a stage of keys is free, for tile i + 1, and one of values.
                // The turn two later cannot pass before this wait, since it takes tile i + 1's keys;
                // at the last tile, which has none to follow, the turn after (S of this tile) serves
                bool ok = i == 0 || turn_done(q_last, base + i - (i + 1 < tiles ? 1 : 0));
                if (!__all_sync(0xffffffffu, ok)) { run = false; break; }
                if (i + 1 < tiles) store_keys();
                // tokens of the block that count: what lies past them may be anything, NaN
                // codes too, and 0 times NaN is not 0.  (Scores of such keys are masked.)
                const int valid = u.hi - token_of(i);
                // A block with a NaN scale makes the weights of the rows that see it NaN; its values
                // must not reach the others, whose weights are 0
                const int finite = vs == vs ? valid : 0;
                if (lane == 0 && kToks * w % kKvBlock == 0)
                    scales[slot * 4 + kToks * w / kKvBlock] =
                        valid > 0 ? make_float4(ks, pow2_log2(vs), pow2_recip_finite(vs), 0.0f) : make_float4(1.0f, 0.0f, 1.0f, 0.0f);
                slot = (slot + 1) % kScaleSlots;
                // the last tile of the item before frees its stage at that item's own barrier, which
                // cannot pass again before this wait: that takes the values of the item's last tile
                ok = !(i == min(1, tiles - 1) && q_before >= 0) || item_done();
                if (!__all_sync(0xffffffffu, ok)) { run = false; break; }
                if (finite < kToks) {
#pragma unroll
                    for (int h = 0; h < kH; ++h)
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            if (r8 + 8 * h >= finite) vraw[h][p] = make_uint4(0u, 0u, 0u, 0u);
                }
                const uint32_t vdst = sbase + T::kOffV + vst * T::kVPanels * T::kPanel;
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint32_t code[4] = {vraw[h][p].x, vraw[h][p].y, vraw[h][p].z, vraw[h][p].w};
                        uint32_t o[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) e4m3x4_to_f16x2(code[j], o[2 * j], o[2 * j + 1]);
                        const uint32_t at = vdst + p * T::kPanel + (kToks * w + 8 * h + r8) * 128;
                        sts128(at + (((2 * c4) ^ r8) << 4), o[0], o[1], o[2], o[3]);
                        sts128(at + (((2 * c4 + 1) ^ r8) << 4), o[4], o[5], o[6], o[7]);
                    }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(T::kVFull) + 8 * vst);
                if (++vst == T::kVStages) vst = 0;
                load_values();                           // of tile i + 1
                load_keys(i + 2, tiles);
            }
            if (tiles > 0) {
#pragma unroll
                for (int q = 0; q < kQt; ++q)
                    if (q < u.live) {
                        turns[q] += tiles + 1;
                        turns_before = turns[q];
                        ++items[q];
                    }
                q_before = q_last;
            }
        }
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------------- products
        // stage and turn of the next keys and values; turns of the score barriers, tiles and
        // items of each query tile so far
        uint32_t kst = 0, kturn = 0, vst = 0, vturn = 0, turns[kQt], pn[kQt], qn[kQt];
#pragma unroll
        for (int q = 0; q < kQt; ++q) turns[q] = pn[q] = qn[q] = 0;
        const uint64_t q0 = desc(sbase, 16), k0 = desc(sbase + T::kOffK, 16), v0 = desc(sbase + T::kOffV, T::kPanel);
        const uint32_t elected = elect_lane();
        Part u;
        bool ok = true;
        for (int k = 0; ok && __all_sync(0xffffffffu, take_part(k, u)); ++k) {
            free_part(k);
            const int tiles = __shfl_sync(0xffffffffu, u.t1 - u.t0, 0), live = __shfl_sync(0xffffffffu, u.live, 0);
            // S of query tile q with the item's next tile of keys, turn n.  It takes the columns that P
            // had two tiles ago, whose product was issued before: the tensor pipe works in the
            // order of issue, whatever the products' kinds.
            //
            // A commit costs the pipe some 50 clocks, so there is one a tile and query tile:
            // after S of tile i (turn i), which says too that every product issued before is done,
            // that with P of tile i - 2 among them.  A turn without scores and a barrier of its own
            // end an item: when P of its last tile but one is used up, and when P of its last is.
            auto scores = [&](int q, uint32_t n) {
                if (q == 0) {
                    if (!__all_sync(0xffffffffu, bar_wait(bar(T::kKFull) + 8 * kst, kturn))) return false;
                }
                fence_after();
                mma_scores<D, 0, 0>(tmem + T::kSCol + (2 * q + (n & 1)) * kKeys, q0 + q * (T::kQBytes >> 4),
                                    k0 + kst * (T::kKPanels * T::kPanel >> 4), elected);
                commit(bar(T::kSFull + 2 * q) + 8 * (n & 1), elected);
                if (q == live - 1) {
                    if (++kst == T::kKStages) { kst = 0; kturn ^= 1; }
                }
                return true;
            };
#pragma unroll
            for (int q = 0; q < kQt; ++q)
                if (ok && q < live && tiles > 0) {
                    ok = __all_sync(0xffffffffu, bar_wait(bar(T::kQFull + q), qn[q]++ & 1));
                    fence_after();
                    ok = ok && scores(q, turns[q]);
                }
            for (int i = 0; ok && i < tiles; ++i) {
#pragma unroll
                for (int q = 0; q < kQt; ++q) {
                    if (!ok || q >= live) break;
                    const uint32_t n = turns[q] + i, p = pn[q]++;
                    if (i + 1 < tiles) {
                        if (!(ok = scores(q, n + 1))) break;
                    } else {
                        commit(bar(T::kSFull + 2 * q) + 8 * ((n + 1) & 1), elected);
                    }
                    ok = (q > 0 || bar_wait(bar(T::kVFull) + 8 * vst, vturn)) &&
                         bar_wait(bar(T::kPFull + 2 * q) + 8 * (p & 1), (p >> 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_after();
                    mma_values<D, 0>(tmem + T::kOCol + q * D, tmem + T::kSCol + (2 * q + (n & 1)) * kKeys,
                                     v0 + vst * (T::kVPanels * T::kPanel >> 4), i > 0 ? 1u : 0u, elected);
                    if (q == live - 1) {
                        if (++vst == T::kVStages) { vst = 0; vturn ^= 1; }
                    }
                    if (i + 1 == tiles) commit(bar(T::kItem + q), elected);
                }
            }
            if (tiles > 0) {
#pragma unroll
                for (int q = 0; q < kQt; ++q)
                    if (q < live) turns[q] += tiles + 1;
            }
        }
        // nothing is in flight when the tensor memory is released
        commit(bar(T::kDone), elected);
        (void)bar_wait(bar(T::kDone), 0);
    } else {
        // ---------------------------------------------------------------------- plan
        long long at = 0, end = 0;                       // of this CTA's share
        bool shares = false;
        if (split) {
            long long all;
            const long long each = share_places<kQt * kRows>(a, gridDim.x, &all);
            shares = each > 0;
            at = min(all, blockIdx.x * each);
            end = min(all, at + each);
        }
        for (int k = 0;; ++k) {
            // every role has the item before, and the loaders are nearly done with it
            if (k >= 1 && !__all_sync(0xffffffffu, bar_wait(bar(T::kPartFree + ((k - 1) & 1)), ((k - 1) >> 1) & 1))) break;
            Part u = {};
            bool found = false, last = false;
            while (!found) {
                if (shares) {
                    if (at >= end) { last = true; break; }
                    const long long first = find_place<kQt * kRows>(a, at, u) + kLead;    // place of tile 0
                    const int tiles = u.t1, full = max(1, tiles);
                    const int t0 = static_cast<int>(max(0ll, at - first)), t1 = static_cast<int>(min(static_cast<long long>(full), end - first));
                    if (u.live == 0) { last = true; break; }
                    u.t0 = t0;
                    u.t1 = min(t1, tiles);
                    if (t0 > 0 || t1 < full) u.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
                    at = first + full;
                    found = t1 > t0;
                } else {
                    unsigned int item = 0;
                    if (lane == 0) item = atomicAdd(a.counters, 1u);
                    item = __shfl_sync(0xffffffffu, item, 0);
                    if (item >= items) { last = true; break; }
                    found = find_unit<kQt * kRows>(a, item, u);
                }
            }
            if (last) u.live = 0;
            if (lane == 0) {
                *const_cast<Part*>(part_at(k)) = u;
                bar_arrive(bar(T::kPartFull + (k & 1)));
            }
            if (last) break;
        }
        // the CTA that leaves last puts the counters back; every planner comes here, by a wait that gave up too
        if (!shares && lane == 0 && atomicAdd(a.counters + 1, 1u) == gridDim.x - 1) {
            a.counters[0] = 0u;
            a.counters[1] = 0u;
        }
    }

    griddep_launch_dependents();
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(T::kCols) : "memory");
    }
}

// The parts of split units, added in their order: a CTA for 32 values of a query tile's
// rows, after the kernel above (whose last CTA would else add a long unit's parts alone).
constexpr int kJoinThreads = 128, kJoinCols = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const __grid_constant__ AttendArgs a, int ctas) {
    using T = Tile<D>;
    __shared__ Part shared_part;
    __shared__ int shared_parts;
    griddep_wait();
    // the unit that CTA blockIdx.x / kQt began last, if others went on with it
    const int qi = blockIdx.x % T::kQt;
    const long long cta = blockIdx.x / T::kQt;
    if (threadIdx.x < 32) {
        long long all;
        Part p = {};
        const long long each = share_places<T::kQt * kRows>(a, ctas, &all);
        const long long begin = min(all, cta * each), end = min(all, begin + each);
        int parts = 0;
        if (end > begin) {
            const long long first = find_place<T::kQt * kRows>(a, end - 1, p) + kLead, past = first + max(1, p.t1);
            if (p.live > qi && first >= begin && first < end && past > end) parts = static_cast<int>((past - 1) / each - cta) + 1;
        }
        if (threadIdx.x == 0) { shared_part = p; shared_parts = parts; }
    }
    __syncthreads();
    const int parts = shared_parts;
    if (parts > 1) {
        const Part& u = shared_part;
        const int row0 = (u.qt * T::kQt + qi) * kRows, rows = min(kRows, u.n * a.group - row0);
        // the first part stands in the second slot of its CTA, the others in the first of theirs
        const size_t step = 2 * T::kQt * T::kPart;
        const float* base = a.partials + (static_cast<size_t>(2 * cta) * T::kQt + qi) * T::kPart;
        const int d = blockIdx.y * kJoinCols + threadIdx.x % 8 * 4;
        for (int row = threadIdx.x / 8; row < rows; row += kJoinThreads / 8) {
            float top = -INFINITY, l = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int p0 = 0; p0 < parts; p0 += 8) {      // eight parts' loads side by side
                float pm[8], pl[8];
                float4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int part = min(p0 + q, parts - 1);
                    const float* from = base + part * step + (part == 0 ? T::kQt * T::kPart : 0);
                    pm[q] = __ldcg(from + D * kRows + row);
                    pl[q] = __ldcg(from + D * kRows + kRows + row);
                    v[q] = __ldcg(reinterpret_cast<const float4*>(from + row * D + d));
                }
                float high = top;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (p0 + q >= parts) pm[q] = -INFINITY;
                    high = fmaxf(high, pm[q]);
                }
                const float ref = high == -INFINITY ? 0.0f : high;
                float f = exp2_approx(top - ref);
                top = high;
                l *= f;
                acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    f = exp2_approx(pm[q] - ref);
                    if (p0 + q >= parts) continue;
                    acc.x = fmaf(v[q].x, f, acc.x); acc.y = fmaf(v[q].y, f, acc.y);
                    acc.z = fmaf(v[q].z, f, acc.z); acc.w = fmaf(v[q].w, f, acc.w);
                    l = fmaf(pl[q], f, l);
                }
            }
            store_row4(a, u.start, u.head, row0 + row, D, d, acc, l);
        }
    }
    griddep_launch_dependents();
}

int unit_rows(int head_dim) { return head_dim <= 128 ? 2 * kRows : kRows; }

// Units that the packed rows can make (their lengths are on the device): a partial tile
// a sequence at most.
long long unit_bound(int tokens, int seqs, int group, int kv_heads, int head_dim) {
    const long long rows = static_cast<long long>(tokens) * group;
    const long long t = rows / unit_rows(head_dim) + seqs;
    return (t < rows ? t : rows) * kv_heads;
}

// Units may be split among the CTAs where they would fill the SMs less than four times.  (Past
// that the second launch and the parts' results cost prompts more than the evenness
// saves: chunks of 4 x 2k tokens, 1024 units, 737 us split and 702 whole.)
bool is_split(long long units, int sms) { return units < 4ll * sms; }

template <int D>
int launch(const AttendArgs& a, long long units, int sms, cudaStream_t stream) {
    using T = Tile<D>;
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(kv_tile_kernel<D>, T::kSmem, opted)) return TRELLIS_ERR_CUDA;
    const bool split = is_split(units, sms);
    const cudaError_t e = launch_programmatic(kv_tile_kernel<D>, static_cast<unsigned>(sms), static_cast<unsigned>(T::kThreads),
                                              T::kSmem, stream, a, split, static_cast<unsigned>(units));
    if (e != cudaSuccess) return TRELLIS_ERR_CUDA;
    if (!split) return TRELLIS_OK;
    return launch_programmatic_grid(kv_join_kernel<D>, dim3(static_cast<unsigned>(sms) * T::kQt, D / kJoinCols), kJoinThreads, 0,
                                    stream, a, sms) == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // namespace

size_t kv_tile_workspace_bytes(int tokens, int seqs, int q_heads, int kv_heads, int head_dim, const DeviceInfo& dev) {
    const long long units = unit_bound(tokens > 0 ? tokens : 1, seqs, q_heads / kv_heads, kv_heads, head_dim);
    if (!is_split(units, dev.num_sms)) return kKvCounterBytes;
    return kKvCounterBytes + static_cast<size_t>(2 * dev.num_sms) * unit_rows(head_dim) * (static_cast<size_t>(head_dim) + 2) * 4;
}

int launch_kv_tile(const AttendArgs& a, int head_dim, const DeviceInfo& dev, cudaStream_t stream) {
    const long long units = unit_bound(a.l.tokens, a.l.seqs, a.group, a.l.kv_heads, head_dim);
    if (units >= (1ll << 31)) return TRELLIS_ERR_SHAPE;
    return head_dim == 64 ? launch<64>(a, units, dev.num_sms, stream)
           : head_dim == 128 ? launch<128>(a, units, dev.num_sms, stream)
                             : launch<256>(a, units, dev.num_sms, stream);
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
