// trellis_lora_add: the low-rank adapters of many requests, added to the output of
// a projection that they share.
//
//   out[m] = bf16( y[m] + s_a * B_a (A_a x[m]) ),  a = the adapter of row m's request
//
// Two launches: h = x A^T (sums over K, the long axis), then out = y + s h B^T (over
// the rank).  Both are skinny: at few rows they read A and B (2 R (K + N) bytes an
// adapter), at many rows x, y and out.  The tensor work is 2 M R (K + 2 N) multiply-adds
// (h counts twice, see below): at m16n8k16's 8 cycles each 32 us of the second kernel's 43
// for its bytes in the largest case below, and about twice that at rank 128 (120 us in all).
//
// Measured (GPU time of both launches; the least bytes at 6.69 TB/s): 1 row, K 5120, N 17408,
// rank 16: 4.6 to 5.1 us, two launches in a row; 64 requests of one row on 24 adapters, K 17408,
// N 5120, rank 32: 17 us (5.7), half of it start and the reads of 64 tiles, which do not
// share an adapter; 4068 rows of 4 requests, K 5120, N 17408, rank 64: 78 us (53), of which
// the first kernel 20 (chain of copy, shared memory and mma of 4 warps an SM) and the second
// 58 at 4.9 TB/s.  Rows without an adapter are copied at 6 TB/s by the same loop.
//
// * The order of a sum's terms is free, so a lane's 8 consecutive elements (16 bytes) serve
//   as its operands of two products, in both factors alike: fragments need no
//   rearrangement.  They come through rings in shared memory that cp.async fills some
//   steps ahead, by whole 128-byte lines.  The two halves of a line change places in odd
//   rows, so that the 16-byte reads (8 rows by 64 bytes a warp) meet no bank conflict.
// * h is summed over K by the warps of a CTA and over K splits by the second kernel,
//   always in the same order.  It stays fp32; the second product takes it as the
//   sum of two bf16 (16 significant bits), so that it rounds far below the one
//   rounding of the result.
// * Rows are cut into tiles inside each request's rows.  A warp of the first kernel takes
//   a tile's 16, 32 or 64 rows by all of the rank and a share of K of its own, so that no
//   two warps read the same.  In the second kernel's tiles of 64 rows the warps, 16 rows
//   each, share B's columns.
// * The first kernel lets the second start once all of its blocks run, after its own wait
//   for what came before: so the second may find its tile and fetch y and B while the
//   first still works, and waits only before it reads h.
#include "kernels.h"
#include "kv_cache.cuh"
#include "trellis.h"

namespace trellis {

namespace {

struct LoraArgs {
    const uint16_t *y, *x, *a, *b;
    const float* scales;         // [adapters]
    const int* starts;           // [segments + 1] rows of each request
    const int* which;            // [segments] adapter, or none where outside 0 .. adapters - 1
    uint16_t* out;
    float* h;                    // [splits][M][R]
    int M, K, N, R, adapters, segments, splits;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes, or zeros (nothing is read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lora_lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void lora_sts(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Segment and rows [row, end) of row tile `tile` (tiles of kTileRows rows, counted
// segment by segment); false past the last one.  Every thread calls it.
template <int kTileRows>
__device__ bool find_tile(const LoraArgs& p, int tile, int* smem, int* seg, int* row, int* end) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int base = 0, got = -1, r = 0, e = 0;
        for (int s0 = 0; s0 < p.segments && got < 0; s0 += 32) {
            const int s = s0 + lane;
            int a = 0, b = 0;
            if (s < p.segments) {
                a = max(0, __ldg(p.starts + s));
                b = min(p.M, __ldg(p.starts + s + 1));
            }
            const int n = b > a ? (b - a + kTileRows - 1) / kTileRows : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const int at = base + incl - n;
            const unsigned hit = __ballot_sync(0xffffffffu, tile >= at && tile < at + n);
            if (hit != 0u) {
                const int src = __ffs(hit) - 1;
                r = __shfl_sync(0xffffffffu, a + (tile - at) * kTileRows, src);
                e = __shfl_sync(0xffffffffu, b, src);
                got = s0 + src;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) { smem[0] = got; smem[1] = r; smem[2] = min(e, r + kTileRows); }
    }
    __syncthreads();
    *seg = smem[0]; *row = smem[1]; *end = smem[2];
    return *seg >= 0;
}

__device__ __forceinline__ int adapter_of(const LoraArgs& p, int seg) {
    const int w = __ldg(p.which + seg);
    return w >= 0 && w < p.adapters ? w : -1;
}

// Offset in a 128-byte line of its 16-byte piece, in row `row`.
__device__ __forceinline__ uint32_t line_piece(int piece, int row) { return (piece ^ ((row & 1) << 2)) * 16; }

// h[split][row][r] = sum over the split's k of x[row][k] a[r][k], for a tile of 16 MT rows
// and a rank of at most 8 NT.  The warps of the CTA, and the splits, share the sum over k
// in slabs of 64: 128 bytes of every row of x and of a, in a ring of the warp's own.
template <int NT, int MT>
struct Down {
    static constexpr int kRows = 16 * MT;
    static constexpr int kStepBytes = (kRows + 8 * NT) * 128;
    static constexpr int kWarps = 4;
    // two CTAs an SM for tiles of 16 rows, which are many; one of the largest
    static constexpr int kFit = (MT == 1 ? 112 : 200) * 1024 / (kWarps * kStepBytes);
    static constexpr int kSteps = kFit < 2 ? 2 : kFit > 4 ? 4 : kFit;
    static constexpr int kRing = kWarps * kSteps * kStepBytes;
    static constexpr int kSums = kWarps * kRows * (8 * NT + 8) * 4;          // [warp][row][R + 8], where the ring was
    static constexpr int kSmem = kRing > kSums ? kRing : kSums;
    static_assert(kSmem <= 232448 - 1024, "shared memory");
};

template <int NT, int MT>
__global__ void __launch_bounds__(Down<NT, MT>::kWarps * 32) lora_down_kernel(const __grid_constant__ LoraArgs p) {
    using S = Down<NT, MT>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int found[4];
    griddep_wait();
    griddep_launch_dependents();
    int seg, row0, end;
    if (!find_tile<S::kRows>(p, blockIdx.x, found, &seg, &row0, &end)) return;
    const int w = adapter_of(p, seg);
    if (w < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint16_t* a = p.a + static_cast<size_t>(w) * p.R * p.K;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::kSteps * S::kStepBytes;
    const int slabs = (p.K + 63) / 64, stride = p.splits * S::kWarps;
    const int sl0 = blockIdx.y * S::kWarps + warp;
    const int crow = lane >> 3, cpiece = lane & 7;       // a copy covers 4 rows by 8 pieces
    const uint32_t mine_at = ring + crow * 128 + line_piece(cpiece, crow);
    const int x_rows = end - row0 - crow, a_rows = p.R - crow;
    const size_t hop = static_cast<size_t>(p.K) * 4;
    const uint16_t* x_at = p.x + static_cast<size_t>(row0 + (x_rows > 0 ? crow : 0)) * p.K;
    const uint16_t* a_at = a + static_cast<size_t>(crow) * p.K;
    auto issue = [&](int sl, int step) {
        const int k = sl * 64 + cpiece * 8;
        const bool in = k < p.K;                         // K is a multiple of 8: a piece is in or out
        const uint32_t dst = mine_at + step * S::kStepBytes;
        const uint16_t *xs = x_at + (in ? k : 0), *as = a_at + (in ? k : 0);
#pragma unroll
        for (int i = 0; i < S::kRows / 4; ++i, xs += hop)        // past the tile's last row anything may stand
            if (4 * i < x_rows) cp_async16_or_zero(dst + i * 512, xs, in);
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i, as += hop)
            if (4 * i < a_rows) cp_async16_or_zero(dst + (S::kRows / 4 + i) * 512, as, in);
    };
    for (int i = 0; i < 2 * NT; ++i)                     // rows past the rank: zero, once
        if (4 * i >= a_rows)
            for (int q = 0; q < S::kSteps; ++q) lora_sts(mine_at + q * S::kStepBytes + (S::kRows / 4 + i) * 512, {0, 0, 0, 0});
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < S::kSteps - 1; ++i) {
        if (sl0 + i * stride < slabs) issue(sl0 + i * stride, i);
        cp_async_commit();
    }
    int step = 0, fill = S::kSteps - 1;
    for (int sl = sl0; sl < slabs; sl += stride) {
        cp_async_wait<S::kSteps - 2>();
        __syncwarp();                                    // the copies of every lane; and its reads of the slot to fill
        const int ahead = sl + (S::kSteps - 1) * stride;
        if (ahead < slabs) issue(ahead, fill);
        cp_async_commit();
        const uint32_t src = ring + step * S::kStepBytes + g * 128;
        step = step + 1 == S::kSteps ? 0 : step + 1;
        fill = fill + 1 == S::kSteps ? 0 : fill + 1;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t at = src + line_piece(4 * q + t, g);
            uint4 u[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) u[i] = lora_lds(at + i * 1024);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint4 b = lora_lds(at + (2 * MT + i) * 1024);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma_bf16(acc[m][i], u[2 * m].x, u[2 * m + 1].x, u[2 * m].y, u[2 * m + 1].y, b.x, b.y);
                    mma_bf16(acc[m][i], u[2 * m].z, u[2 * m + 1].z, u[2 * m].w, u[2 * m + 1].w, b.z, b.w);
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();                                     // every warp is done with its ring
    // 8 floats between rows: 4 rows of a half warp's pairs fall into different banks
    const int pitch = p.R + 8;
    float* sums = reinterpret_cast<float*>(smem);
    float* mine = sums + warp * S::kRows * pitch;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int c = 8 * i + 2 * t;
            if (c < p.R) {
                *reinterpret_cast<float2*>(mine + (16 * m + g) * pitch + c) = make_float2(acc[m][i][0], acc[m][i][1]);
                *reinterpret_cast<float2*>(mine + (16 * m + g + 8) * pitch + c) = make_float2(acc[m][i][2], acc[m][i][3]);
            }
        }
    __syncthreads();
    const int quads = p.R / 4, live = (end - row0) * quads;
    float* h = p.h + (static_cast<size_t>(blockIdx.y) * p.M + row0) * p.R;
    for (int e = threadIdx.x; e < live; e += S::kWarps * 32) {
        const int row = e / quads, at = row * pitch + (e - row * quads) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < S::kWarps; ++q) {
            const float4 s = *reinterpret_cast<const float4*>(sums + q * S::kRows * pitch + at);
            v.x += s.x; v.y += s.y; v.z += s.z; v.w += s.w;
        }
        *reinterpret_cast<float4*>(h + static_cast<size_t>(e) * 4) = v;
    }
}

// out = y + s h B^T for a tile of 16 RG rows, a warp's 16 rows by 64 columns at a step.
// RG warps share the step's B; RG = 1: each warp has columns of its own.  NS: slabs of 32
// of the rank.
template <int NS, int RG, bool kVec>
struct Up {
    static constexpr int kWarps = RG == 1 ? 4 : RG;
    static constexpr int kCols = 64 * (kWarps / RG);                         // of the CTA's warps in a step
    static constexpr int kB = 64 * NS * 64, kY = kVec ? 16 * 128 : 0;
    static constexpr int kStepBytes = kB * (kWarps / RG) + kY * kWarps;
    static constexpr int kCtas = RG == 1 ? 2 : 4;                           // an SM
    static constexpr int kFit = 224 / kCtas * 1024 / kStepBytes;
    static constexpr int kSteps = kFit < 2 ? 2 : kFit > 4 ? 4 : kFit;
    static constexpr int kSmem = kSteps * kStepBytes;
    static_assert(kSmem <= 232448 - 1024, "shared memory");
};

template <int NS, int RG, bool kVec>
__global__ void __launch_bounds__(Up<NS, RG, kVec>::kWarps * 32, Up<NS, RG, kVec>::kCtas)
lora_up_kernel(const __grid_constant__ LoraArgs p, int cols_per_cta) {
    using S = Up<NS, RG, kVec>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int found[4];
    int seg, row0, end;
    if (!find_tile<16 * RG>(p, blockIdx.x, found, &seg, &row0, &end)) {
        griddep_wait();                                  // what follows may rely on what came before this kernel
        return;
    }
    const int w = adapter_of(p, seg);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rg = warp % RG, cg = warp / RG;
    const int wrow = row0 + rg * 16;                     // the warp's rows: it may have none
    const int ra = wrow + g, rb = ra + 8;
    const bool la = ra < end, lb = rb < end;
    const uint16_t* B = p.b + (w >= 0 ? static_cast<size_t>(w) * p.N * p.R : 0);
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const uint32_t ring_b = base + cg * S::kB, ring_y = base + S::kB * (S::kWarps / RG) + warp * S::kY;
    const int c_end = min(p.N, (static_cast<int>(blockIdx.y) + 1) * cols_per_cta);
    const int first = blockIdx.y * cols_per_cta + cg * 64;
    const int crow = lane >> 3, cpiece = lane & 7;
    auto sync = [] {
        if constexpr (RG == 1) __syncwarp();
        else __syncthreads();
    };
    // B: a copy covers kBRows of its rows, which are NS 64 bytes each; odd ones have the halves of their lines exchanged
    constexpr int kBRows = RG * 8 / NS;
    const int bn = (rg * 32 + lane) / (4 * NS), bpiece = (rg * 32 + lane) % (4 * NS);
    const uint32_t b_at = ring_b + bn * (NS * 64) + (NS == 1 ? bpiece * 16 : line_piece(bpiece, bn));
    const bool b_have = w >= 0 && bpiece * 8 < p.R;
    const uint16_t* b_from = B + static_cast<size_t>(bn) * p.R + bpiece * 8;
    const size_t b_hop = static_cast<size_t>(kBRows) * p.R;
    // y: 4 rows by 8 pieces
    const uint32_t y_at = ring_y + crow * 128 + line_piece(cpiece, crow);
    const int y_rows = end - wrow - crow;
    const size_t y_from = static_cast<size_t>(wrow + crow) * p.N + cpiece * 8, y_hop = static_cast<size_t>(p.N) * 4;
    auto issue = [&](int c0, int step) {
        if (b_have) {
            const uint32_t dst = b_at + step * S::kStepBytes;
            const uint16_t* src = b_from + static_cast<size_t>(c0) * p.R;
            const int left = p.N - c0 - bn;              // past the last column anything may stand
#pragma unroll
            for (int i = 0; i < 64 / kBRows; ++i, src += b_hop)
                if (i * kBRows < left) cp_async16_or_zero(dst + i * kBRows * NS * 64, src, true);
        }
        if constexpr (kVec) {
            const uint32_t dst = y_at + step * S::kStepBytes;
            const uint16_t* src = p.y + y_from + c0;
            const int rows = c0 + cpiece * 8 < p.N ? y_rows : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i, src += y_hop)
                if (4 * i < rows) cp_async16_or_zero(dst + i * 512, src, true);
        }
    };
    if (bpiece * 8 >= p.R)                               // past the rank: zero, once
        for (int q = 0; q < S::kSteps; ++q)
            for (int i = 0; i < 64 / kBRows; ++i) lora_sts(b_at + q * S::kStepBytes + i * kBRows * NS * 64, {0, 0, 0, 0});
    constexpr int kHop = S::kCols;
#pragma unroll
    for (int i = 0; i < S::kSteps - 1; ++i) {
        if (first + i * kHop < c_end) issue(first + i * kHop, i);
        cp_async_commit();
    }
    const float s = w >= 0 ? __ldg(p.scales + w) : 0.0f;
    griddep_wait();
    // h as the sum of two bf16: fragments hi, lo of 2 products a slab
    uint32_t hi[NS][2][4], lo[NS][2][4];
#pragma unroll
    for (int sl = 0; sl < NS; ++sl) {
        const int r = sl * 32 + t * 8;
        float v[2][8];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
        if (w >= 0 && r < p.R) {
#pragma unroll 4
            for (int sp = 0; sp < p.splits; ++sp) {
                const float* h = p.h + static_cast<size_t>(sp) * p.M * p.R + r;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q == 0 ? la : lb) {
                        const float4* h4 = reinterpret_cast<const float4*>(h + static_cast<size_t>(q == 0 ? ra : rb) * p.R);
                        const float4 f0 = h4[0], f1 = h4[1];
                        v[q][0] += f0.x; v[q][1] += f0.y; v[q][2] += f0.z; v[q][3] += f0.w;
                        v[q][4] += f1.x; v[q][5] += f1.y; v[q][6] += f1.z; v[q][7] += f1.w;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float v0 = s * v[q][2 * i], v1 = s * v[q][2 * i + 1];
                const uint32_t h2 = pack_bf16x2(v0, v1);
                // product i / 2; registers: row g then row g + 8, first pair then second.
                // An infinite sum has no rest (inf - inf would make it NaN)
                const float e0 = v0 - bf16_lo(h2), e1 = v1 - bf16_hi(h2);
                hi[sl][i >> 1][(i & 1) * 2 + q] = h2;
                lo[sl][i >> 1][(i & 1) * 2 + q] = pack_bf16x2(e0 == e0 ? e0 : 0.0f, e1 == e1 ? e1 : 0.0f);
            }
    }
    int step = 0, fill = S::kSteps - 1;
    for (int c0 = first; c0 < c_end; c0 += kHop) {
        cp_async_wait<S::kSteps - 2>();
        sync();                                          // every copy of the step; and all are done with the slot to fill
        const int ahead = c0 + (S::kSteps - 1) * kHop;
        if (ahead < c_end) issue(ahead, fill);
        cp_async_commit();
        const uint32_t src_b = ring_b + step * S::kStepBytes, src_y = ring_y + step * S::kStepBytes;
        step = step + 1 == S::kSteps ? 0 : step + 1;
        fill = fill + 1 == S::kSteps ? 0 : fill + 1;
        if (wrow >= end) continue;
        // column c0 + 32 q + 8 t + 2 i + e belongs to tile i, so a lane's columns are 8 neighbours
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
            if (w >= 0) {
#pragma unroll
                for (int sl = 0; sl < NS; ++sl)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 32 * q + 8 * (g >> 1) + 2 * i + (g & 1), piece = sl * 4 + t;
                        const uint4 b = lora_lds(src_b + n * (NS * 64) + (NS == 1 ? piece * 16 : line_piece(piece, g)));
                        mma_bf16(acc[i], lo[sl][0][0], lo[sl][0][1], lo[sl][0][2], lo[sl][0][3], b.x, b.y);
                        mma_bf16(acc[i], lo[sl][1][0], lo[sl][1][1], lo[sl][1][2], lo[sl][1][3], b.z, b.w);
                        mma_bf16(acc[i], hi[sl][0][0], hi[sl][0][1], hi[sl][0][2], hi[sl][0][3], b.x, b.y);
                        mma_bf16(acc[i], hi[sl][1][0], hi[sl][1][1], hi[sl][1][2], hi[sl][1][3], b.z, b.w);
                    }
            }
            if constexpr (kVec) {
                // y's piece gives way to the result's; without an adapter y passes, whatever its bits
                if (w >= 0) {
                    const uint32_t at = src_y + g * 128 + line_piece(4 * q + t, g);
                    const uint4 ya = lora_lds(at), yb = lora_lds(at + 1024);
                    const uint32_t y0[4] = {ya.x, ya.y, ya.z, ya.w}, y1[4] = {yb.x, yb.y, yb.z, yb.w};
                    uint32_t o0[4], o1[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o0[i] = pack_bf16x2(bf16_lo(y0[i]) + acc[i][0], bf16_hi(y0[i]) + acc[i][1]);
                        o1[i] = pack_bf16x2(bf16_lo(y1[i]) + acc[i][2], bf16_hi(y1[i]) + acc[i][3]);
                    }
                    lora_sts(at, o0);
                    lora_sts(at + 1024, o1);
                }
            } else {
                const int col = c0 + 32 * q + 8 * t;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = col + 2 * i + e;
                        if (c >= p.N) continue;
                        if (la) {
                            const size_t at = static_cast<size_t>(ra) * p.N + c;
                            const uint16_t v = p.y[at];
                            p.out[at] = w < 0 ? v : bf16_bits_rn(bf16_bits_to_f32(v) + acc[i][e]);
                        }
                        if (lb) {
                            const size_t at = static_cast<size_t>(rb) * p.N + c;
                            const uint16_t v = p.y[at];
                            p.out[at] = w < 0 ? v : bf16_bits_rn(bf16_bits_to_f32(v) + acc[i][2 + e]);
                        }
                    }
            }
        }
        if constexpr (kVec) {
            __syncwarp();
            const uint32_t src = src_y + crow * 128 + line_piece(cpiece, crow);
            uint16_t* dst = p.out + y_from + c0;
            const int rows = c0 + cpiece * 8 < p.N ? y_rows : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i, dst += y_hop)
                if (4 * i < rows) *reinterpret_cast<uint4*>(dst) = lora_lds(src + i * 512);
        }
    }
    cp_async_wait<0>();
    griddep_launch_dependents();
}

struct LoraShape {
    bool wide;                       // tiles of many rows
    int down_tiles, splits;          // of the first kernel: tiles are an upper bound, the lengths are on the device
    int up_tiles, cols;              // of the second: columns of a CTA
};

// NT of the first kernel: eighths of the rank, rounded up to what is compiled.
int down_nt(int R) { return R <= 16 ? 2 : R <= 32 ? 4 : R <= 64 ? 8 : 16; }

template <int NT>
void down_size(bool wide, int* rows, int* warps, int* steps) {
    using W = Down<NT, NT == 16 ? 2 : 4>;
    using F = Down<NT, 1>;
    *rows = wide ? W::kRows : F::kRows;
    *warps = wide ? W::kWarps : F::kWarps;
    *steps = wide ? W::kSteps : F::kSteps;
}

LoraShape lora_shape(int M, int K, int N, int R, int segments, const DeviceInfo& dev) {
    LoraShape s;
    // Large tiles read an adapter once for all of their rows, but there are few of them, and
    // short segments leave them half empty.  Measured, us with large tiles / with 16 rows
    // (K = N = 5120): rank 64, 4 segments of 128 rows 20.5 / 11.6, of 256 24.7 / 21.6, of 512
    // 27.6 / 35.0, 16 of 128 30.5 / 35.0, 64 of 64 52.7 / 47.9; rank 16, 4 of 256 12.8 / 12.9,
    // of 512 20.5 / 23.2, 64 of 64 34.1 / 30.9; rank 128, 4 of 128 32.0 / 29.1, of 256
    // 29.1 / 42.8, 64 of 64 64.9 / 101.5.
    s.wide = R > 64 ? M > 512 && M / segments >= 48 : M > 1024 && M / segments >= 96;
    auto tiles = [&](int rows) {     // at most one partial tile a segment, and no tile without a row
        const long long bound = static_cast<long long>(M) / rows + segments;
        return static_cast<int>(bound < M ? bound : M);
    };
    int rows, warps, steps;
    switch (down_nt(R)) {
        case 2: down_size<2>(s.wide, &rows, &warps, &steps); break;
        case 4: down_size<4>(s.wide, &rows, &warps, &steps); break;
        case 8: down_size<8>(s.wide, &rows, &warps, &steps); break;
        default: down_size<16>(s.wide, &rows, &warps, &steps); break;
    }
    s.down_tiles = tiles(rows);
    s.up_tiles = tiles(s.wide ? 64 : 16);
    // K is split until the CTAs fill the SMs, or each warp's first copies cover its share:
    // more splits would only be more to add up
    const int slabs = (K + 63) / 64;
    const int fill = (s.wide ? 1 : 2) * dev.num_sms / s.down_tiles;
    const int most = (slabs + warps * (steps - 1) - 1) / (warps * (steps - 1));
    const int splits = fill < most ? fill : most;
    s.splits = splits < 1 ? 1 : splits > 32 ? 32 : splits;
    const int unit = s.wide ? 64 : 256;                  // columns of a CTA's warps in a step
    const int col_units = (N + unit - 1) / unit;
    // Ragged tiles of many rows even out in shorter turns: 4k rows by 17408 columns, rank 64,
    // 75 us (both kernels) at twice what is resident, 80 at four times.  Of 16-row tiles one
    // wave is best (64 rows: 19 us; 23 at 10 CTAs an SM).
    int parts = ((s.wide ? 8 : 2) * dev.num_sms + s.up_tiles - 1) / s.up_tiles;
    parts = parts < col_units ? parts : col_units;
    s.cols = (col_units + parts - 1) / parts * unit;
    return s;
}

template <int NT, int MT>
cudaError_t launch_down(const LoraArgs& p, const LoraShape& s, cudaStream_t stream) {
    using S = Down<NT, MT>;
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(lora_down_kernel<NT, MT>, S::kSmem, opted)) return cudaErrorInvalidValue;
    return launch_programmatic_grid(lora_down_kernel<NT, MT>, dim3(s.down_tiles, s.splits), S::kWarps * 32, S::kSmem, stream, p);
}

template <int NS, int RG, bool kVec>
cudaError_t launch_up_as(const LoraArgs& p, const LoraShape& s, cudaStream_t stream) {
    using S = Up<NS, RG, kVec>;
    static std::atomic<unsigned long long> opted{0};
    if (!smem_opt_in(lora_up_kernel<NS, RG, kVec>, S::kSmem, opted)) return cudaErrorInvalidValue;
    return launch_programmatic_grid(lora_up_kernel<NS, RG, kVec>, dim3(s.up_tiles, (p.N + s.cols - 1) / s.cols), S::kWarps * 32,
                                    S::kSmem, stream, p, s.cols);
}

template <int NS>
cudaError_t launch_up(const LoraArgs& p, const LoraShape& s, bool vec, cudaStream_t stream) {
    if (s.wide) return vec ? launch_up_as<NS, 4, true>(p, s, stream) : launch_up_as<NS, 4, false>(p, s, stream);
    return vec ? launch_up_as<NS, 1, true>(p, s, stream) : launch_up_as<NS, 1, false>(p, s, stream);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_lora_sizes(int M, int K, int N, int R, int adapters, int segments) {
    if (M < 0 || K < 1 || N < 1 || R < 1 || adapters < 1 || segments < 1 || K % 8 != 0 || R % 8 != 0)
        return TRELLIS_ERR_SHAPE;
    if (R > 128 || M > 65536 || segments > 65536) return TRELLIS_ERR_UNSUPPORTED;
    return TRELLIS_OK;
}

}  // namespace

}  // namespace trellis

extern "C" {

int trellis_lora_add_workspace_size(int M, int K, int N, int R, int adapters, int segments, size_t* bytes) {
    using namespace trellis;
    if (bytes == nullptr) return TRELLIS_ERR_NULL;
    int rc = check_lora_sizes(M, K, N, R, adapters, segments);
    if (rc != TRELLIS_OK) return rc;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    const LoraShape s = lora_shape(M > 0 ? M : 1, K, N, R, segments, dev);
    // the products' counter region stays free (and zero) in front
    *bytes = (size_t(1) << 20) + static_cast<size_t>(s.splits) * M * R * 4;
    return TRELLIS_OK;
}

int trellis_lora_add(const uint16_t* y, const uint16_t* x, const uint16_t* a, const uint16_t* b, const float* scales,
                     const int* starts, const int* which, int M, int K, int N, int R, int adapters, int segments,
                     uint16_t* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace trellis;
    if (y == nullptr || x == nullptr || a == nullptr || b == nullptr || scales == nullptr || starts == nullptr ||
        which == nullptr || out == nullptr)
        return TRELLIS_ERR_NULL;
    int rc = check_lora_sizes(M, K, N, R, adapters, segments);
    if (rc != TRELLIS_OK) return rc;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(y, 2) || !aligned(out, 2) ||
        !aligned(scales, 4) || !aligned(starts, 4) || !aligned(which, 4))
        return TRELLIS_ERR_ALIGN;
    size_t need = 0;
    rc = trellis_lora_add_workspace_size(M, K, N, R, adapters, segments, &need);
    if (rc != TRELLIS_OK) return rc;
    if (workspace == nullptr || workspace_bytes < need) return TRELLIS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return TRELLIS_ERR_ALIGN;
    if (M == 0) return TRELLIS_OK;
    DeviceInfo dev;
    rc = device_info(dev);
    if (rc != TRELLIS_OK) return rc;
    const LoraShape s = lora_shape(M, K, N, R, segments, dev);
    LoraArgs p;
    p.y = y; p.x = x; p.a = a; p.b = b; p.scales = scales; p.starts = starts; p.which = which; p.out = out;
    p.h = reinterpret_cast<float*>(static_cast<char*>(workspace) + (size_t(1) << 20));
    p.M = M; p.K = K; p.N = N; p.R = R; p.adapters = adapters; p.segments = segments; p.splits = s.splits;
    cudaError_t e = cudaSuccess;
    switch (down_nt(R)) {
        case 2: e = s.wide ? launch_down<2, 4>(p, s, stream) : launch_down<2, 1>(p, s, stream); break;
        case 4: e = s.wide ? launch_down<4, 4>(p, s, stream) : launch_down<4, 1>(p, s, stream); break;
        case 8: e = s.wide ? launch_down<8, 4>(p, s, stream) : launch_down<8, 1>(p, s, stream); break;
        default: e = s.wide ? launch_down<16, 2>(p, s, stream) : launch_down<16, 1>(p, s, stream); break;
    }
    if (e != cudaSuccess) return TRELLIS_ERR_CUDA;
    // 16-byte accesses of y and out
    const bool vec = N % 8 == 0 && aligned(y, 16) && aligned(out, 16);
    e = R <= 32 ? launch_up<1>(p, s, vec, stream) : R <= 64 ? launch_up<2>(p, s, vec, stream)
                                                            : launch_up<4>(p, s, vec, stream);
    return e == cudaSuccess ? TRELLIS_OK : TRELLIS_ERR_CUDA;
}

}  // extern "C"
