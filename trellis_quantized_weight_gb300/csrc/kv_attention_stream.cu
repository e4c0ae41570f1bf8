// Attention over the paged 8-bit cache for few query rows: the form for single
// tokens and short drafts.
//
//   out[i] = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * q_i . k_j),
//   over the cached tokens j that row i sees (pos_i - window < j <= pos_i).
//
// What bounds it: 2 D bytes of codes a cached token and key head, each read once
// and used by the head group's few rows, so HBM.  Measured at D = 128, 8 key heads (GPU time;
// the least bytes at 6.69 TB/s): one sequence of 131071 tokens 55 us (40); 64 of 1 to 16384
// 172 us (153), 6.0 TB/s, at about 7.5 TB/s between the start (5 us of dependent first loads)
// and the joins; one of 777 tokens 8.5 us (0.2), which is start and joins alone.  With 9
// to 16 rows a unit the products' instructions take over: 16 x 300 to 9000 tokens, 8 rows
// 43 us, 16 rows 59.  Everything else is arranged around a long stream of 16-byte loads:
//
// * Work: a unit is (sequence, NT * 8 query rows of one key head's group, key
//   head); its tokens are cut into tiles of 16 tokens a warp.  All units' tiles
//   in a row are dealt to the CTAs in equal contiguous shares, whatever the
//   lengths, so a CTA holds at most two pieces of units that others share.  The
//   pieces' sums meet in the workspace; the CTA that finishes last adds them in
//   CTA order (the same order on every run).
// * Loads: each warp copies the codes of its steps (whole lines of the cache) into a
//   ring of its own in shared memory (cp.async), several steps ahead, in the order in
//   which its lanes will read them.  No barrier wider than a warp is in the loop.
// * Products: S^T = K Q^T and O^T = V^T P^T on m16n8k16 with f16 operands and fp32
//   sums.  e4m3 -> f16 is exact.  The order of a sum's terms is free, so a lane's 16
//   consecutive bytes of a key serve as its operand of four products, the query
//   fragments being loaded in the same order; the values of two tokens are paired
//   by byte permutes.  Keys take the 16-row side, so a group of up to 8 rows
//   pays for 8.  (These products are a few per cent of the tensor rate: at 2 D bytes
//   a token the legacy matrix instruction is far from being the limit.)
// * Scales: a power of two times a score is exact.  The key block's scale multiplies
//   the scores; the value block's is added to them as its log2, so that
//   p' = p * v_scale comes out of the exponential and no further multiplication
//   is needed; the denominators add p' / v_scale.
// * Running maximum: p' is taken against a reference that is only moved when a score
//   exceeds it by 2^15.5, so a step has one vote instead of reductions.  p' in f16 (11
//   significant bits down to 2^-14, 2^-25 of error below) is the one rounding between q, k, v and
//   the fp32 sums.  A weight that rounds to 0 still counts in the denominators, so the
//   reference is set 2^7 below the largest score: 2^17 tokens lose under 2^-15 of the
//   largest weight (2^-8 with the reference at the largest score).  Queries enter as f16 times a
//   power of two per row: bf16's 8 bits down to 2^-17 of the row's largest, 2^-25 of it below.
#include <cfloat>

#include "kv_attention.cuh"
#include "trellis.h"

namespace trellis {

namespace {

// The reference moves when exceeded by 2^15.5 (f16 ends at 65504), to the largest score over 2^7: the
// weights that vanish in f16, under 2^-25, are under 2^-32 of the largest then.
constexpr float kMoveBy = 15.5f;
constexpr float kBelow = 7.0f;
constexpr int kJoin = 16;                // pieces of a unit that one CTA joins

// Warps of a CTA and ring steps by head width and rows: 128 to 160 KB of codes in
// flight an SM beside the warps' sums.
template <int D, int NT> struct StreamShape;
template <int NT> struct StreamShape<64, NT> { static constexpr int kWarps = 8, kSteps = 8; };
template <> struct StreamShape<128, 1> { static constexpr int kWarps = 8, kSteps = 5; };
template <> struct StreamShape<128, 2> { static constexpr int kWarps = 8, kSteps = 4; };
template <int NT> struct StreamShape<256, NT> { static constexpr int kWarps = 6, kSteps = 3; };

template <int D, int NT>
struct Stream {
    static constexpr int kWarps = StreamShape<D, NT>::kWarps;
    static constexpr int kSteps = StreamShape<D, NT>::kSteps;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * NT;                 // query rows of a unit
    static constexpr int kTile = kKvBlock * kWarps;      // cached tokens of a tile
    static constexpr int kStepBytes = 2 * kKvBlock * D;  // codes of one warp's step
    static constexpr int kRing = kWarps * kSteps * kStepBytes;
    static constexpr int kScaleOff = kRing;              // [warps][steps][2] floats
    static constexpr int kPart = kRows * D + 2 * kRows;  // floats of a partial result: O [rows][D], m, l
    static constexpr int kSumsOff = kScaleOff + kWarps * kSteps * 8;
    static constexpr int kMiscOff = kSumsOff + kWarps * kPart * 4;
    static constexpr int kSmem = kMiscOff + 256;
    static_assert(kSmem <= 232448, "shared memory");
};

struct Unit {
    int seq, head, qt;        // query tile
    Seq s;
    int lo, hi;               // cached tokens [lo, hi) that its rows see (lo a multiple of 16)
    int tiles;
};

// A unit costs a CTA at least about as much as streaming kMinTiles tiles (its warps'
// sums meet, its result is stored), so a shorter one counts as that many in the
// shares: tile k of a unit stands at its unit's first place + lead + k.
constexpr int kMinTiles = 3;
__device__ __forceinline__ int lead_of(int tiles) { return tiles < kMinTiles ? kMinTiles - tiles : 0; }

// Quotient of two counts of places: 32 bits wide but for enormous batches.
__device__ __forceinline__ long long div_places(long long x, long long y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// Equal shares of `all` places: the first `rest` of the CTAs hold one more.
struct Shares {
    long long each, rest;
    __device__ __forceinline__ Shares(long long all, long long ctas) {
        each = div_places(all, ctas);
        rest = all - each * ctas;
    }
    __device__ __forceinline__ long long first(long long cta) const { return cta * each + min(cta, rest); }
    __device__ __forceinline__ long long holder(long long place) const {
        const long long wide = rest * (each + 1);
        return place < wide ? div_places(place, each + 1) : rest + div_places(place - wide, each);
    }
};

// Tiles of a query tile, and its token range.
template <int D, int NT>
__device__ __forceinline__ int unit_tiles(const AttendArgs& a, const Seq& s, int qt, int* lo, int* hi) {
    using S = Stream<D, NT>;
    const int first = qt * S::kRows / a.group, last = min(s.n - 1, (qt * S::kRows + S::kRows - 1) / a.group);
    *hi = max(0, min(s.total, s.p0 + last + 1));
    const int low = a.window > 0 ? max(0, s.p0 + first + 1 - a.window) : 0;
    *lo = low & ~(kKvBlock - 1);
    const int span = *hi - *lo;
    return span > 0 ? (span + S::kTile - 1) / S::kTile : 1;   // an empty unit still writes its zeros
}

template <int D, int NT>
__device__ long long seq_places(const AttendArgs& a, const Seq& s) {
    if (s.n <= 0) return 0;
    const int qts = (s.n * a.group + Stream<D, NT>::kRows - 1) / Stream<D, NT>::kRows;
    long long sum = 0;
    int lo, hi;
    for (int qt = 0; qt < qts; ++qt) sum += max(kMinTiles, unit_tiles<D, NT>(a, s, qt, &lo, &hi));
    return sum * a.l.kv_heads;                             // places
}

// A walk over units in their order: heads, then query tiles, then sequences.
template <int D, int NT>
struct Walk {
    Unit u;
    Seq ahead;                // sequence u.seq + 1, loaded before it is needed

    __device__ __forceinline__ void begin(const AttendArgs& a, const Unit& first) {
        u = first;
        ahead = load_seq(a.l, min(u.seq + 1, a.l.seqs - 1));
    }
    // The caller knows that there is a unit after this one.
    __device__ __forceinline__ void next(const AttendArgs& a) {
        if (++u.head < a.l.kv_heads) return;               // the same rows and tokens
        u.head = 0;
        if (++u.qt * Stream<D, NT>::kRows >= u.s.n * a.group) {
            u.qt = 0;
            do {
                u.seq = min(u.seq + 1, a.l.seqs - 1);
                u.s = ahead;
                ahead = load_seq(a.l, min(u.seq + 1, a.l.seqs - 1));
            } while (u.s.n <= 0 && u.seq < a.l.seqs - 1);
        }
        u.tiles = unit_tiles<D, NT>(a, u.s, u.qt, &u.lo, &u.hi);
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(Stream<D, NT>::kThreads, 1) kv_stream_kernel(const __grid_constant__ AttendArgs a) {
    using S = Stream<D, NT>;
    constexpr int KJ = D / 64;                  // 16-byte pieces of a key row a lane
    constexpr int VJ = D >= 128 ? D / 128 : 1;  // pieces of a value row a lane (8 bytes at D = 64)
    constexpr int MT = D / 16;                  // 16-row tiles of O^T
    constexpr int kCopies = D / 32;             // 16-byte copies of a lane for the keys of a step (values alike)
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    griddep_wait();

    // ---- this CTA's share of all units' tiles -------------------------------------------
    // prefix sums over the sequences, a contiguous chunk a thread
    long long* scan = reinterpret_cast<long long*>(smem + S::kMiscOff);
    const int per = (a.l.seqs + S::kThreads - 1) / S::kThreads;
    const int s0 = min(a.l.seqs, static_cast<int>(threadIdx.x) * per), s1 = min(a.l.seqs, s0 + per);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) mine += seq_places<D, NT>(a, load_seq(a.l, s));
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
    }
    const long long ctas = min(static_cast<long long>(gridDim.x), all);
    const long long cta = blockIdx.x;
    if (cta >= ctas) { griddep_launch_dependents(); return; }
    const Shares shares(all, ctas);
    const long long begin = shares.first(cta), end = shares.first(cta + 1);
    // the thread whose sequences hold place `begin` finds the unit
    Unit* found = reinterpret_cast<Unit*>(smem + S::kMiscOff + 8 * S::kWarps);
    int* found_off = reinterpret_cast<int*>(found + 1);
    long long at = before + incl - mine;
    if (begin >= at && begin < at + mine) {
        Unit f;
        f.seq = s0;
        f.s = load_seq(a.l, s0);
        long long c = seq_places<D, NT>(a, f.s);
        while (begin >= at + c) {
            at += c;
            f.s = load_seq(a.l, ++f.seq);
            c = seq_places<D, NT>(a, f.s);
        }
        long long off = begin - at;
        f.qt = 0;
        f.tiles = unit_tiles<D, NT>(a, f.s, 0, &f.lo, &f.hi);
        while (off >= static_cast<long long>(max(kMinTiles, f.tiles)) * a.l.kv_heads) {
            off -= static_cast<long long>(max(kMinTiles, f.tiles)) * a.l.kv_heads;
            f.tiles = unit_tiles<D, NT>(a, f.s, ++f.qt, &f.lo, &f.hi);
        }
        const int places = max(kMinTiles, f.tiles);
        f.head = static_cast<int>(div_places(off, places));
        *found = f;
        *found_off = static_cast<int>(off - static_cast<long long>(f.head) * places);
    }
    __syncthreads();

    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::kSteps * S::kStepBytes;
    const uint32_t ring_sc = static_cast<uint32_t>(__cvta_generic_to_shared(smem + S::kScaleOff)) + warp * S::kSteps * 8;
    float* sums = reinterpret_cast<float*>(smem + S::kSumsOff);
    int* ticket = reinterpret_cast<int*>(smem + S::kMiscOff);
    float* joined = reinterpret_cast<float*>(smem + S::kMiscOff + 64);     // [2][rows]

    // ---- copies: a walk of its own, steps ahead of the sums and across units ---------------
    // The 16 tokens of a step lie one after another, so copy r of a lane is bytes
    // 512 r + 16 lane of them: whole lines of the cache.  Where its 16 bytes go in the
    // ring makes them the operands of the lane that reads there; the exclusive ors keep
    // both the copies and the reads free of bank conflicts.
    auto k_slot = [&](int r) {
        const int chunk = r * 32 + lane, tok = chunk / (D / 16), c = chunk % (D / 16);
        const int j = c >> 2;                   // token = row 8 h + g, chunk t + 4 j
        return ((tok >> 3) * KJ + j) * 512 + ((((tok & 7) * 4 + (c & 3)) ^ ((j & 1) * 4)) * 16);
    };
    auto v_slot = [&](int r) {
        const int chunk = r * 32 + lane, tok = chunk / (D / 16), c = chunk % (D / 16);
        const int vt = (tok & 7) >> 1, vr = (tok & 1) + ((tok >> 3) << 1);   // token 2 t + (r & 1) + 8 (r >> 1)
        if constexpr (D == 64) return vr * 256 + vt * 64 + ((c ^ (vt & 2)) * 16);
        return (vr * VJ + (c >> 3)) * 512 + vt * 128 + (((c & 7) ^ (2 * vt)) * 16);
    };
    const int shift = a.l.page_shift - 4;       // blocks of a page, log2
    Walk<D, NT> ahead;
    ahead.begin(a, *found);
    long long ahead_base = begin - *found_off;  // first place of the walk's unit
    int ahead_tile = max(0, *found_off - lead_of(ahead.u.tiles));
    // this warp's next block; -1: none is left.  Starts the load of its page id.
    auto seek = [&](int& blk, int& page, int& head) {
        blk = -1;
        while (true) {
            if (ahead_base + lead_of(ahead.u.tiles) + ahead_tile >= end) return;
            if (ahead_tile == ahead.u.tiles) {
                ahead_base += max(kMinTiles, ahead.u.tiles);
                if (ahead_base >= end) return;
                ahead.next(a);
                ahead_tile = 0;
                continue;
            }
            const int b = ahead.u.lo / kKvBlock + ahead_tile * S::kWarps + warp;
            ++ahead_tile;
            if (b * kKvBlock < ahead.u.hi) {
                blk = b;
                head = ahead.u.head;
                page = kv_page(a.l, ahead.u.seq, b >> shift);
                // and of the line that the ids of the steps to come lie in
                const int later = min((b >> shift) + 32, a.l.page_cols - 1);
                asm volatile("prefetch.global.L1 [%0];"
                             :: "l"(a.l.pages + static_cast<size_t>(ahead.u.seq) * a.l.page_cols + later));
                return;
            }
        }
    };
    auto issue = [&](int slot, int blk, int page, int head) {
        if (blk < 0) return;
        const int in_page = blk & ((1 << shift) - 1);
        const size_t unit = static_cast<size_t>(page) * a.l.kv_heads + head;
        const size_t off = (unit * a.l.page_size + in_page * kKvBlock) * D + lane * 16;
        const uint32_t dst = ring + slot * S::kStepBytes;
#pragma unroll
        for (int r = 0; r < kCopies; ++r) {
            cp_async16(dst + k_slot(r), a.k_codes + off + r * 512);
            cp_async16(dst + kKvBlock * D + v_slot(r), a.v_codes + off + r * 512);
        }
        const size_t sc = unit * (a.l.page_size / kKvBlock) + in_page;
        if (lane < 2) cp_async4(ring_sc + slot * 8 + lane * 4, (lane == 0 ? a.k_scales : a.v_scales) + sc);
    };
    int next_blk, next_page = 0, next_head = 0;
    seek(next_blk, next_page, next_head);
#pragma unroll 1
    for (int i = 0; i < S::kSteps - 1; ++i) {   // the page ids are neighbours: one miss serves most
        issue(i, next_blk, next_page, next_head);
        cp_async_commit();
        if (next_blk >= 0) seek(next_blk, next_page, next_head);
    }
    int slot = 0, fill = S::kSteps - 1;         // ring slots read and filled next

    // ---- queries of a unit: raw, loaded a unit ahead ----------------------------------------
    Walk<D, NT> walk;
    walk.begin(a, *found);
    long long base = begin - *found_off;        // first place of the unit
    int tile0 = max(0, *found_off - lead_of(walk.u.tiles));
    uint4 raw[NT][KJ][2];
    auto load_queries = [&](const Unit& u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = u.qt * S::kRows + nt * 8 + g;
            const int tok = r / a.group;
            const bool live = tok < u.s.n;
            const uint4* row = reinterpret_cast<const uint4*>(
                a.q + static_cast<size_t>(u.s.start + (live ? tok : 0)) * a.q_stride +
                (static_cast<size_t>(u.head) * a.group + r % a.group) * D);
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    raw[nt][j][h] = live ? row[2 * (t + 4 * j) + h] : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load_queries(walk.u);

    while (base < end) {
        const Unit u = walk.u;
        // the unit's tiles that stand before this CTA's end; none where only its lead does
        const int tile1 = static_cast<int>(min(static_cast<long long>(u.tiles), end - base - lead_of(u.tiles)));
        if (tile1 <= tile0) break;

        // f16 fragments, each row times a power of two
        uint32_t qf[NT][4 * KJ][2];
        float qmul[NT][2];                      // of this lane's two columns (rows 2t, 2t + 1 of each 8)
        int limit[NT][2], lower[NT][2];         // cached tokens [lower, limit) that they see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t most = 0u;
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w[4] = {raw[nt][j][h].x, raw[nt][j][h].y, raw[nt][j][h].z, raw[nt][j][h].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) most = max(most, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                }
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int e = query_exponent(most);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w[4] = {raw[nt][j][h].x, raw[nt][j][h].y, raw[nt][j][h].z, raw[nt][j][h].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        qf[nt][4 * j + 2 * h + (i >> 1)][i & 1] = f32_to_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
                }
            // the column's factor, from the lane that holds its row
            // (a row with an infinity or a NaN has no softmax: it is NaN, whatever signs its scores would get)
            const float up = most >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                             : __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                qmul[nt][h] = __shfl_sync(0xffffffffu, up, (2 * t + h) * 4);
                const int tk = min((u.qt * S::kRows + nt * 8 + 2 * t + h) / a.group, u.s.n - 1);
                limit[nt][h] = min(u.hi, u.s.p0 + tk + 1);
                lower[nt][h] = a.window > 0 ? u.s.p0 + tk + 1 - a.window : 0;
            }
        }
        // tokens that every row sees
        const int all_hi = min(u.hi, u.s.p0 + u.qt * S::kRows / a.group + 1);
        const int all_lo = a.window > 0
            ? u.s.p0 + min((u.qt * S::kRows + S::kRows - 1) / a.group, u.s.n - 1) + 1 - a.window : 0;
        const long long unit_base = base;
        base += max(kMinTiles, u.tiles);
        if (base < end) {
            walk.next(a);
            load_queries(walk.u);
        }

        float o[NT][MT][4];
        float m[NT][2], sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
            m[nt][0] = m[nt][1] = -INFINITY;
            sum[nt][0] = sum[nt][1] = 0.0f;
        }

        for (int tile = tile0; tile < tile1; ++tile) {
            const int tok0 = u.lo + (tile * S::kWarps + warp) * kKvBlock;
            if (tok0 >= u.hi) break;            // the walk of the copies passes over it too
            __syncwarp();                       // every lane has read the slot that is filled now
            issue(fill, next_blk, next_page, next_head);
            if (next_blk >= 0) seek(next_blk, next_page, next_head);
            cp_async_commit();
            cp_async_wait<S::kSteps - 1>();
            __syncwarp();                       // every lane's copies have landed
            const uint32_t src = ring + slot * S::kStepBytes;
            float ks, vs;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(ring_sc + slot * 8) : "memory");
            slot = slot + 1 == S::kSteps ? 0 : slot + 1;
            fill = fill + 1 == S::kSteps ? 0 : fill + 1;

            // scores: two chains of products
            float sc[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[nt][h][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                const uint4 ka = lds128(src + j * 512 + ((lane ^ ((j & 1) * 4)) * 16));
                const uint4 kb = lds128(src + (KJ + j) * 512 + ((lane ^ ((j & 1) * 4)) * 16));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16x2(wa[w], a0, a2);
                    e4m3x4_to_f16x2(wb[w], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(sc[nt][w & 1], a0, a1, a2, a3, qf[nt][4 * j + w][0], qf[nt][4 * j + w][1]);
                }
            }
            const float lv = pow2_log2(vs), iv = pow2_recip_finite(vs);
            const bool edge = tok0 + kKvBlock > all_hi || tok0 < all_lo;
            // A NaN value scale makes the weights of the rows that see its block NaN (lv is).  Its values
            // must not reach rows that do not see it, whose weights are 0
            const int values_end = edge && vs != vs ? tok0 : u.hi;
            bool over = false;
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int h = j & 1;
                    x[nt][j] = fmaf(sc[nt][0][j] + sc[nt][1][j], qmul[nt][h] * ks, lv);
                    if (edge) {
                        const int tok = tok0 + g + (j >> 1) * 8;
                        if (tok >= limit[nt][h] || tok < lower[nt][h]) x[nt][j] = -INFINITY;
                    }
                    over |= x[nt][j] > m[nt][h] + kMoveBy;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float top = fmaxf(x[nt][h], x[nt][h + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        top = fmaxf(top - kBelow, m[nt][h]);
                        const float f = m[nt][h] == -INFINITY ? 0.0f : exp2_approx(m[nt][h] - top);
                        m[nt][h] = top;
                        sum[nt][h] *= f;
#pragma unroll
                        for (int q = 0; q < MT; ++q) { o[nt][q][h] *= f; o[nt][q][h + 2] *= f; }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
                const float m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
                const float p0 = exp2_approx(x[nt][0] - m0), p1 = exp2_approx(x[nt][1] - m1);
                const float p2 = exp2_approx(x[nt][2] - m0), p3 = exp2_approx(x[nt][3] - m1);
                sum[nt][0] = fmaf(p0 + p2, iv, sum[nt][0]);
                sum[nt][1] = fmaf(p1 + p3, iv, sum[nt][1]);
                pf[nt][0] = movmatrix_trans(f32_to_f16x2(p0, p1));
                pf[nt][1] = movmatrix_trans(f32_to_f16x2(p2, p3));
            }
            // slots past the last token may hold anything, NaN too: their values count as 0, as those of a
            // block with a NaN scale do (0 times NaN is not 0)
            const bool tail = tok0 + kKvBlock > values_end;
            const uint32_t vsrc = src + kKvBlock * D;
            auto products = [&](int q, const uint32_t (&w)[4]) {       // 4 values of 4 tokens: tiles 2q, 2q + 1
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h == 0 ? 0x5140u : 0x7362u;
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16x2(__byte_perm(w[0], w[1], sel), a0, a1);
                    e4m3x4_to_f16x2(__byte_perm(w[2], w[3], sel), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * q + h], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            };
            bool keep[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) keep[r] = !tail || tok0 + 2 * t + (r & 1) + (r >> 1) * 8 < values_end;
            if constexpr (D == 64) {
                uint32_t w[2][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint2 v = lds64(vsrc + r * 256 + t * 64 + ((g >> 1) ^ (t & 2)) * 16 + (g & 1) * 8);
                    w[0][r] = keep[r] ? v.x : 0u;
                    w[1][r] = keep[r] ? v.y : 0u;
                }
                products(0, w[0]);
                products(1, w[1]);
            } else {
#pragma unroll
                for (int j = 0; j < VJ; ++j) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint4 v = lds128(vsrc + (r * VJ + j) * 512 + t * 128 + (g ^ (2 * t)) * 16);
                        w[0][r] = keep[r] ? v.x : 0u;
                        w[1][r] = keep[r] ? v.y : 0u;
                        w[2][r] = keep[r] ? v.z : 0u;
                        w[3][r] = keep[r] ? v.w : 0u;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) products(4 * j + q, w[q]);
                }
            }
        }

        // ---- the warps' sums meet (the copies of the next unit are under way) ---------------
        {
            float* mine_o = sums + warp * S::kPart;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float l = sum[nt][h];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    const int row = nt * 8 + 2 * t + h;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        // tile i, row g: the value index that load and permute gave it
                        const int d = D == 64 ? 8 * g + 2 * i : (g + 8 * (i / 8)) * 16 + 2 * (i % 8);
                        *reinterpret_cast<float2*>(mine_o + row * D + d) = make_float2(o[nt][i][h], o[nt][i][h + 2]);
                    }
                    if (g == 0) {
                        mine_o[S::kRows * D + row] = m[nt][h];
                        mine_o[S::kRows * D + S::kRows + row] = l;
                    }
                }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == u.tiles;
        // where the unit's pieces go: CTA c's slot 2c when the unit began before it, else 2c + 1
        float* piece = a.partials + (2 * cta + (tile0 == 0 ? 1 : 0)) * S::kPart;
        const int rows = min(S::kRows, u.s.n * a.group - u.qt * S::kRows);
        for (int e = threadIdx.x * 4; e < rows * D; e += S::kThreads * 4) {
            const int row = e / D, d = e % D;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) top = fmaxf(top, sums[w * S::kPart + S::kRows * D + row]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float l = 0.0f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) {
                const float* p = sums + w * S::kPart;
                const float f = exp2_approx(p[S::kRows * D + row] - ref);
                const float4 v = *reinterpret_cast<const float4*>(p + row * D + d);
                acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
                l = fmaf(p[S::kRows * D + S::kRows + row], f, l);
            }
            if (whole) {
                store_row4(a, u.s.start, u.head, u.qt * S::kRows + row, D, d, acc, l);
            } else {
                *reinterpret_cast<float4*>(piece + row * D + d) = acc;
                if (d == 0) {
                    piece[S::kRows * D + row] = top;
                    piece[S::kRows * D + S::kRows + row] = l;
                }
            }
        }
        if (!whole) {
            // the CTAs that hold the unit's first and last tile
            const long long c0 = shares.holder(unit_base + lead_of(u.tiles));
            const int pieces = static_cast<int>(shares.holder(unit_base + lead_of(u.tiles) + u.tiles - 1) - c0) + 1;
            // Groups of kJoin pieces are joined by their last CTA into the slot of their first
            // piece, and the groups by the last of those: the order of the sums is always the
            // same, and a long sequence's many pieces are not one CTA's chain of loads.
            auto part = [&](int p) { return a.partials + (2 * (c0 + p) + (p == 0 ? 1 : 0)) * S::kPart; };
            auto last_of = [&](unsigned int* counter, int of) {
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) {
                    const unsigned int got = atomicAdd(counter, 1u);
                    *ticket = got == static_cast<unsigned int>(of - 1);
                    if (*ticket) *counter = 0u;                  // left ready for the next call
                }
                __syncthreads();
                const bool yes = *ticket != 0;
                if (yes) __threadfence();
                return yes;
            };
            // joins pieces from, from + step, ... below to; `final` stores the unit's rows
            auto join = [&](int from, int to, int step, bool final) {
                for (int e = threadIdx.x * 4; e < rows * D; e += S::kThreads * 4) {
                    const int row = e / D, d = e % D;
                    float top = -INFINITY, l = 0.0f;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
                    for (int p0 = from; p0 < to; p0 += 8 * step) {
                        float pm[8], pl[8];
                        float4 v[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const int p = p0 + q * step;
                            const float* src = part(p < to ? p : from);
                            pm[q] = __ldcg(src + S::kRows * D + row);
                            pl[q] = __ldcg(src + S::kRows * D + S::kRows + row);
                            v[q] = __ldcg(reinterpret_cast<const float4*>(src + e));
                        }
                        float high = top;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (p0 + q * step >= to) pm[q] = -INFINITY;
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
                            if (p0 + q * step >= to) continue;
                            acc.x = fmaf(v[q].x, f, acc.x); acc.y = fmaf(v[q].y, f, acc.y);
                            acc.z = fmaf(v[q].z, f, acc.z); acc.w = fmaf(v[q].w, f, acc.w);
                            l = fmaf(pl[q], f, l);
                        }
                    }
                    if (final) {
                        store_row4(a, u.s.start, u.head, u.qt * S::kRows + row, D, d, acc, l);
                        continue;
                    }
                    // the row's maximum and denominator in its first piece are still read by the
                    // other threads of the row: they are replaced below, from shared memory
                    *reinterpret_cast<float4*>(part(from) + e) = acc;
                    if (d == 0) { joined[row] = top; joined[S::kRows + row] = l; }
                }
                if (!final) {
                    __syncthreads();
                    if (threadIdx.x < 2 * S::kRows) part(from)[S::kRows * D + threadIdx.x] = joined[threadIdx.x];
                }
            };
            const int mine_p = static_cast<int>(cta - c0);
            if (pieces <= kJoin) {
                if (last_of(a.counters + 2 * c0 + 1, pieces)) join(0, pieces, 1, true);
            } else {
                const int first = mine_p / kJoin * kJoin, to = min(first + kJoin, pieces);
                if (last_of(a.counters + 2 * (c0 + first) + (first == 0 ? 1 : 0), to - first)) {
                    join(first, to, 1, false);
                    if (last_of(a.counters + 2 * (gridDim.x + c0), (pieces + kJoin - 1) / kJoin))
                        join(0, pieces, kJoin, true);
                }
            }
        }
        __syncthreads();                        // the sums are read before the next unit's are stored
        tile0 = 0;
    }
    cp_async_wait<0>();
    griddep_launch_dependents();
}

template <int D, int NT>
int launch(const AttendArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    using S = Stream<D, NT>;
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(kv_stream_kernel<D, NT>, S::kSmem, opted)) return TRELLIS_ERR_CUDA;
    const cudaError_t e = launch_programmatic(kv_stream_kernel<D, NT>, static_cast<unsigned>(dev.num_sms),
                                              static_cast<unsigned>(S::kThreads), S::kSmem, stream, a);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

// Rows of a unit: 16 where a sequence has more than 8 rows to a key head, except
// at D = 256, whose sums for 16 rows do not fit the registers.
bool two_tiles(int head_dim, int rows) { return rows > 8 && head_dim < 256; }

}  // namespace

size_t kv_stream_workspace_bytes(int head_dim, int rows, const DeviceInfo& dev) {
    const size_t unit_rows = two_tiles(head_dim, rows) ? 16 : 8;
    return kKvCounterBytes + static_cast<size_t>(dev.num_sms) * 2 * (unit_rows * head_dim + 2 * unit_rows) * 4;
}

int launch_kv_stream(const AttendArgs& a, int head_dim, int rows, const DeviceInfo& dev, cudaStream_t stream) {
    const bool two = two_tiles(head_dim, rows);
    if (head_dim == 64) return two ? launch<64, 2>(a, dev, stream) : launch<64, 1>(a, dev, stream);
    if (head_dim == 128) return two ? launch<128, 2>(a, dev, stream) : launch<128, 1>(a, dev, stream);
    return launch<256, 1>(a, dev, stream);
}

}  // namespace trellis
